// Products of 8-bit activations (or gradients) with the 8-bit frozen weight,
// for gfx950:
//
//   forward    y_tj  = sum_k x_tk W_jk,   contraction over in;
//   backward   dx_tk = sum_j g_tj W_jk,   contraction over out,
//
// every operand an e4m3 value times its block's power of two (q8_common.hpp).
// The scaled matrix instruction mfma_scale_f32_32x32x64_f8f6f4 takes one
// exponent byte per operand row and 32 contraction steps and multiplies by both
// powers of two itself; a block of 128 is then four times the same byte, and no
// vector instruction is spent between blocks.  Sums are fp32, rounded once.
//
// Inside the instruction, the eight products of eight consecutive steps are cut
// (towards zero) to multiples of 2^-13 times the power of two of the largest
// one's operand exponents before they are added; between groups of eight it
// keeps 24 bits and more.  Measured with p beside 448 * 448 - 448 * 448: p is
// cut to a multiple of 2^3 in their group, kept down to 2^-8 in the next.  Over
// 8192 steps of normal or heavy-tailed values that is 1.5e-5 to 6.5e-5 of the
// sum's norm, a fifteenth to a quarter of fp16's rounding of the result and
// below a twentieth of bf16's, next to the 2^-4 of each operand's own rounding:
// the price taken for the instruction's rate, twice the 16-bit one's.
//
// Kernels:
//   q8_gemm_tile    a workgroup owns a BM x BN tile of the output and a range
//                   of the contraction's stages of 128.  Stages go global ->
//                   LDS by DMA into a ring; fragments are read one half stage
//                   ahead of the matrix instructions that use them, one read
//                   between two instructions, so the matrix pipe is fed without
//                   a pause by one wave per SIMD.  The backward's weight panel
//                   keeps its rows (the contraction axis) and is transposed by
//                   the reads (ds_read_b64_tr_b8);
//   q8_gemm_join    adds the fp32 tiles of a split contraction in order;
//   q8_gemm_few     few rows: the weight is streamed once, straight from global
//                   memory into the fragments of mfma 16x16x128.
#include <algorithm>
#include <type_traits>

#include "dma_common.hpp"
#include "q8_common.hpp"

namespace dora {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// ds_read_b64_tr_b8: in each group of 16 lanes, source lane L gives the address
// of 8 consecutive bytes of row L/2 (half L%2 of 16 columns); result lane i
// receives column i of the 8 rows, row 0 in its lowest byte.  As the other
// fragment reads, the result is valid after lds_wait().
template <int OFF>
__device__ inline u32x2 lds_read_tr8_at(uint32_t base) {
  static_assert(OFF >= 0 && OFF < 65536, "ds offset field");
  u32x2 v;
  asm volatile("ds_read_b64_tr_b8 %0, %1 offset:%2" : "=v"(v) : "v"(base), "n"(OFF) : "memory");
  return v;
}
template <int OFF>
__device__ inline uint32_t lds_read4_at(uint32_t base) {
  static_assert(OFF >= 0 && OFF < 65536, "ds offset field");
  uint32_t v;
  asm volatile("ds_read_b32 %0, %1 offset:%2" : "=v"(v) : "v"(base), "n"(OFF) : "memory");
  return v;
}
__device__ inline void tie2(u32x2& v) { asm volatile("" : "+v"(v)); }

// f(0), f(1), .. f(N - 1) with compile-time arguments.
template <class F, int... I>
__device__ inline void unrolled(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ inline void unrolled(F&& f) {
  unrolled(static_cast<F&&>(f), std::make_integer_sequence<int, N>{});
}

// Tile geometry: WM x WN waves, each TMW x TNW matrix tiles of 32 x 32 with
// their accumulators in registers; a ring of NS stages of 128 contraction
// steps.
//
// LDS images.  X and the forward's W panel: rows of 128 bytes, logical 16-byte
// chunk c of row p in slot c ^ ((p/2) % 8): 16 consecutive rows at one chunk
// then fall in 16 distinct bank groups.  The backward's W panel: 128 rows of BN
// bytes; a transposing read touches 8 consecutive rows and two chunks c, c + 1
// (c even), so the chunk is exchanged by the row, leaving its lowest bit alone,
// which spreads the 16 (row, chunk) pairs over the 16 bank groups.
template <int WM_, int WN_, int TMW_, int TNW_, int NS_, bool TRANS_>
struct Q8Tile {
  static constexpr int WM = WM_, WN = WN_, TMW = TMW_, TNW = TNW_, NS = NS_;
  static constexpr bool TRANS = TRANS_;
  static constexpr int NW = WM * WN, NT = 64 * NW;
  static constexpr int BM = 32 * TMW * WM, BN = 32 * TNW * WN, BK = 128;
  static constexpr int X_BYTES = BM * BK, W_BYTES = BN * BK, STAGE_BYTES = X_BYTES + W_BYTES;
  static constexpr int XQ = X_BYTES / 1024 / NW, WQ = W_BYTES / 1024 / NW, L = XQ + WQ;  // DMA instructions a wave
  static constexpr int E_BYTES = BM * 4;  // exponents of the X rows, four stages
  static constexpr int LDS_BYTES = NS * STAGE_BYTES + 2 * E_BYTES;
  static constexpr int CPR = BN / 16;  // chunks per row of the backward's W panel
  static_assert(X_BYTES % (1024 * NW) == 0 && W_BYTES % (1024 * NW) == 0, "whole DMA instructions per wave");
  static_assert(NW % 2 == 0 && BM % 64 == 0, "panel swizzle and exponent DMA");
  static_assert(BN == 128 || BN == 256, "the backward's panel rows");
  static_assert((32 * TNW) % 32 == 0 && 128 % (32 * TNW) == 0, "a wave's columns lie in one weight block");
  static_assert(NS >= 2 && NS <= 4, "an exponent slot is not overwritten before its four stages are done");
  static_assert(LDS_BYTES <= 160 * 1024, "LDS");
};

struct GemmArgs {
  const uint8_t *xq, *xe, *wq, *we;
  int64_t T, N;      // output rows and columns
  int64_t xp, wp;    // bytes of a row of xq and wq
  int64_t xep, wep;  // bytes of a row of exponents
  int64_t wrows;     // rows of wq (whole tiles)
  int S;             // stages of the contraction
  int nRB, nTiles, nSplit;
  uint32_t group;
  void* y;
  int vec;  // 16-byte stores of y
  float* part;
};

// Rows of y from a wave's accumulators: register q of lane l is output column
// 8*(q/4) + 4*(l/32) + q%4 of its tile, row l%32.  Packed in pairs, two groups
// of four columns change places between the lane halves, and each lane then
// holds 8 consecutive columns.
template <int DT>
__device__ inline void store_tile(const GemmArgs& a, int64_t t, int64_t c0, const f32x16& acc, int half) {
  using T16 = typename Dt<DT>::T;
  typedef T16 t2 __attribute__((ext_vector_type(2)));
  uint32_t p[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    p[i] = __builtin_bit_cast(uint32_t, t2{Dt<DT>::from_f(acc[2 * i]), Dt<DT>::from_f(acc[2 * i + 1])});
#pragma unroll
  for (int g = 0; g < 2; ++g) {
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      auto s = __builtin_amdgcn_permlane32_swap(p[4 * g + d], p[4 * g + 2 + d], false, false);
      p[4 * g + d] = s[0];
      p[4 * g + 2 + d] = s[1];
    }
  }
  if (t >= a.T) return;
  T16* y = static_cast<T16*>(a.y) + t * a.N;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int64_t c = c0 + 16 * g + 8 * half;
    const u32x4 w = u32x4{p[4 * g], p[4 * g + 1], p[4 * g + 2], p[4 * g + 3]};
    if (a.vec) {
      if (c < a.N) *reinterpret_cast<u32x4*>(y + c) = w;
    } else {
      const auto v = __builtin_bit_cast(typename Dt<DT>::V8, w);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < a.N) y[c + i] = v[i];
    }
  }
}

// Tile order: groups of `group` column tiles, row blocks within a group, on
// XCD-contiguous ranges: an XCD's concurrent tiles form a block of rows and
// columns whose panels its L2 holds for all of them.
__device__ inline void tile_of(uint32_t v, const GemmArgs& a, int& rb, int& nt) {
  const uint32_t nRB = static_cast<uint32_t>(a.nRB), nTl = static_cast<uint32_t>(a.nTiles), G = a.group;
  const uint32_t grp = v / (G * nRB);
  const uint32_t gn = min(G, nTl - grp * G);
  const uint32_t loc = v - grp * G * nRB;
  rb = static_cast<int>(loc / gn);
  nt = static_cast<int>(grp * G + loc % gn);
}

template <int DT, class TL>
__global__ __launch_bounds__(TL::NT, 1) void q8_gemm_tile(GemmArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[TL::LDS_BYTES];
  const uint32_t v = static_cast<uint32_t>(xcd_logical_index());
  const uint32_t tiles = static_cast<uint32_t>(a.nRB) * static_cast<uint32_t>(a.nTiles);
  if (v >= tiles * static_cast<uint32_t>(a.nSplit)) return;
  const int sp = static_cast<int>(v / tiles);
  int rb, nt;
  tile_of(v - static_cast<uint32_t>(sp) * tiles, a, rb, nt);
  const int64_t m0 = static_cast<int64_t>(rb) * TL::BM, n0 = static_cast<int64_t>(nt) * TL::BN;
  const int st0 = static_cast<int>(static_cast<int64_t>(a.S) * sp / a.nSplit);
  const int st1 = static_cast<int>(static_cast<int64_t>(a.S) * (sp + 1) / a.nSplit);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / TL::WN, wn = wave % TL::WN;
  const int frow = lane & 31, half = lane >> 5;
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_char_t*)smem));

  // Buffer resources over the tile's rows; rows past the operand read zero.
  auto rsrc = [](const uint8_t* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), static_cast<short>(0), static_cast<int>(bytes),
                                             kBufferWord3);
  };
  const int64_t xrows = min(a.T - m0, static_cast<int64_t>(TL::BM));
  const __amdgpu_buffer_rsrc_t rx = rsrc(a.xq + m0 * a.xp, xrows * a.xp);
  const __amdgpu_buffer_rsrc_t re = rsrc(a.xe + m0 * a.xep, xrows * a.xep);
  const int64_t wr = TL::TRANS ? 0 : min(a.wrows - n0, static_cast<int64_t>(TL::BN));
  const __amdgpu_buffer_rsrc_t rw = TL::TRANS ? rx : rsrc(a.wq + n0 * a.wp, wr * a.wp);

  const __amdgpu_buffer_rsrc_t none = rsrc(a.xq, 0);

  // Per-lane DMA offsets.  Instruction q of wave w moves 1 KiB block q*NW + w of
  // its panel, lane l writing bytes 16l .. 16l + 15.
  const int xr = wave * 8 + (lane >> 3);
  const uint32_t kc = static_cast<uint32_t>(((lane & 7) ^ ((xr >> 1) & 7)) * 16);
  const uint32_t xo = static_cast<uint32_t>(xr * a.xp) + kc;
  const uint32_t xstep = static_cast<uint32_t>(TL::NW * 8 * a.xp);
  uint32_t wo, wstep;
  if constexpr (TL::TRANS) {
    constexpr int RPI = 64 / TL::CPR;  // rows per instruction
    const int r = wave * RPI + lane / TL::CPR, sl = lane % TL::CPR;
    // (row + q*NW*RPI has the same swizzle: NW*RPI is a multiple of 8)
    static_assert((TL::NW * RPI) % 8 == 0, "swizzle period");
    const int c = sl ^ (TL::CPR == 16 ? 2 * (r & 7) : 2 * ((r >> 1) & 3));
    const int64_t col = n0 + 16 * c;
    wo = col < a.wp ? static_cast<uint32_t>(r * a.wp + col) : kOob;
    wstep = col < a.wp ? static_cast<uint32_t>(TL::NW * RPI * a.wp) : 0u;
  } else {
    wo = static_cast<uint32_t>(xr * a.wp) + kc;
    wstep = static_cast<uint32_t>(TL::NW * 8 * a.wp);
  }
  // one DMA instruction of a stage (k = 0 .. L - 1, compile time)
  auto issue1 = [&](int st, int slot, auto kk) {
    constexpr int k = decltype(kk)::value;
    char* so = smem + slot * TL::STAGE_BYTES;
    const bool in = st < st1;
    if constexpr (k < TL::XQ) {
      dma16(in ? rx : none, so + (k * TL::NW + wave) * 1024, xo + k * xstep + static_cast<uint32_t>(st) * TL::BK);
    } else {
      constexpr int q = k - TL::XQ;
      char* d = so + TL::X_BYTES + (q * TL::NW + wave) * 1024;
      if constexpr (TL::TRANS) {
        const __amdgpu_buffer_rsrc_t rs =
            rsrc(a.wq + static_cast<int64_t>(st) * TL::BK * a.wp, in ? TL::BK * a.wp : 0);
        dma16(rs, d, wo + q * wstep);
      } else {
        dma16(in ? rw : none, d, wo + q * wstep + static_cast<uint32_t>(st) * TL::BK);
      }
    }
  };
  // Exponents of the X rows, one dword (four stages) a row, before the first of
  // the stages it serves; stage groups are counted from stage 0 of the operand.
  auto issue_exp = [&](int st) {
    if (TL::BM / 64 > wave) {
      char* d = smem + TL::NS * TL::STAGE_BYTES + ((st >> 2) & 1) * TL::E_BYTES + wave * 256;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(st < st1 ? re : none, (lds_void_t*)d, 4,
                                               static_cast<uint32_t>((wave * 64 + lane) * a.xep) + (st & ~3), 0, 0, 0);
    }
  };
  static_assert(TL::BM / 64 <= TL::NW, "one exponent DMA instruction a wave");
  auto issue_all = [&](int st, int slot) {
    if (st == st0 || (st & 3) == 0) issue_exp(st);
    unrolled<TL::L>([&](auto kk) { issue1(st, slot, kk); });
  };

  // Fragment read addresses within a stage slot: half stage s, lane half h takes
  // contraction steps 64s + 32h .. + 31.  (The instruction's own order of the
  // contraction steps within a lane does not matter: both operands use the same.)
  const int sw = (frow >> 1) & 7;
  uint32_t co[2][2];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int c = 0; c < 2; ++c) co[s][c] = static_cast<uint32_t>(((4 * s + 2 * half + c) ^ sw) * 16);
  const uint32_t xrow = lds0 + static_cast<uint32_t>((wm * TL::TMW * 32 + frow) * TL::BK);
  const uint32_t wrow = lds0 + static_cast<uint32_t>(TL::X_BYTES + (wn * TL::TNW * 32 + frow) * TL::BK);
  const uint32_t erow = lds0 + static_cast<uint32_t>(TL::NS * TL::STAGE_BYTES + (wm * TL::TMW * 32 + frow) * 4);
  uint32_t wtr[TL::TNW];
  if constexpr (TL::TRANS) {
    const int L16 = lane & 15, g = lane >> 4;
    const int r = 32 * half + (L16 >> 1);  // + 64 s + 8 piece: the swizzle sees only r % 8
    const int f = TL::CPR == 16 ? 2 * (r & 7) : 2 * ((r >> 1) & 3);
#pragma unroll
    for (int j = 0; j < TL::TNW; ++j) {
      const int c = (wn * TL::TNW + j) * 2 + (g & 1);
      wtr[j] = lds0 + static_cast<uint32_t>(TL::X_BYTES + r * TL::BN + ((c ^ f) * 16) + (L16 & 1) * 8);
    }
  }

  f32x16 acc[TL::TMW][TL::TNW];
#pragma unroll
  for (int i = 0; i < TL::TMW; ++i)
#pragma unroll
    for (int j = 0; j < TL::TNW; ++j) acc[i][j] = f32x16{};

  // A half stage's fragments: X rows as two 16-byte reads, W as two (forward)
  // or four transposing reads.
  struct Frag {
    u32x4 x[TL::TMW][2];
    u32x4 w[TL::TRANS ? 1 : TL::TNW][2];
    u32x2 t[TL::TRANS ? TL::TNW : 1][4];
  };
  constexpr int NR = 2 * TL::TMW + (TL::TRANS ? 4 : 2) * TL::TNW;  // reads of a half stage
  // read n of half stage s (n, s compile time)
  auto read1 = [&](Frag& f, uint32_t so, auto ss, auto nn) {
    constexpr int s = decltype(ss)::value, n = decltype(nn)::value;
    if constexpr (n < 2 * TL::TMW) {
      constexpr int i = n / 2, c = n % 2;
      f.x[i][c] = lds_read16_at<i * 32 * TL::BK>(xrow + co[s][c] + so);
    } else if constexpr (!TL::TRANS) {
      constexpr int j = (n - 2 * TL::TMW) / 2, c = n % 2;
      f.w[j][c] = lds_read16_at<j * 32 * TL::BK>(wrow + co[s][c] + so);
    } else {
      constexpr int j = (n - 2 * TL::TMW) / 4, p = (n - 2 * TL::TMW) % 4;
      f.t[j][p] = lds_read_tr8_at<(64 * s + 8 * p) * TL::BN>(wtr[j] + so);
    }
  };
  auto tie_all = [&](Frag& f) {
#pragma unroll
    for (int i = 0; i < TL::TMW; ++i)
#pragma unroll
      for (int c = 0; c < 2; ++c) tie(f.x[i][c]);
    if constexpr (TL::TRANS) {
#pragma unroll
      for (int j = 0; j < TL::TNW; ++j)
#pragma unroll
        for (int p = 0; p < 4; ++p) tie2(f.t[j][p]);
    } else {
#pragma unroll
      for (int j = 0; j < TL::TNW; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c) tie(f.w[j][c]);
    }
  };
  uint32_t sx[TL::TMW];  // exponent bytes of the current stage (lowest byte)
  uint32_t swb = 0;      // the wave's weight block's
  auto mfma1 = [&](const Frag& f, int i, int j) {
    const v8i xv = {static_cast<int>(f.x[i][0][0]), static_cast<int>(f.x[i][0][1]), static_cast<int>(f.x[i][0][2]),
                    static_cast<int>(f.x[i][0][3]), static_cast<int>(f.x[i][1][0]), static_cast<int>(f.x[i][1][1]),
                    static_cast<int>(f.x[i][1][2]), static_cast<int>(f.x[i][1][3])};
    v8i wv;
    if constexpr (TL::TRANS) {
      wv = v8i{static_cast<int>(f.t[j][0][0]), static_cast<int>(f.t[j][0][1]), static_cast<int>(f.t[j][1][0]),
               static_cast<int>(f.t[j][1][1]), static_cast<int>(f.t[j][2][0]), static_cast<int>(f.t[j][2][1]),
               static_cast<int>(f.t[j][3][0]), static_cast<int>(f.t[j][3][1])};
    } else {
      wv = v8i{static_cast<int>(f.w[j][0][0]), static_cast<int>(f.w[j][0][1]), static_cast<int>(f.w[j][0][2]),
               static_cast<int>(f.w[j][0][3]), static_cast<int>(f.w[j][1][0]), static_cast<int>(f.w[j][1][1]),
               static_cast<int>(f.w[j][1][2]), static_cast<int>(f.w[j][1][3])};
    }
    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wv, xv, acc[i][j], 0, 0, 0, static_cast<int>(swb), 0,
                                                                static_cast<int>(sx[i]));
  };
  constexpr int NM = TL::TMW * TL::TNW;  // matrix instructions of a half stage
  // The weight block's exponent byte of a stage (a scalar load: the address is
  // the wave's own and nothing writes there while the kernel runs).
  typedef const uint32_t __attribute__((address_space(4))) const_u32;
  const int64_t wblk = (n0 + wn * TL::TNW * 32) / kQ8Block;
  const int64_t nblk = (TL::TRANS ? a.wp : a.wrows) / kQ8Block;
  const int64_t wb = min(wblk, nblk - 1);  // columns past the weight have zero panels: any exponent
  auto wexp_idx = [&](int st) { return TL::TRANS ? static_cast<int64_t>(st) * a.wep + wb : wb * a.wep + st; };
  auto wexp_load = [&](int st) -> uint32_t {
    return ((const_u32*)(reinterpret_cast<uintptr_t>(a.we)))[wexp_idx(st) >> 2];
  };
  // The stage's exponent dwords of this lane's rows.
  uint32_t ex[TL::TMW];
  auto read_exp = [&](int st) {
    const uint32_t ea = erow + static_cast<uint32_t>(((st >> 2) & 1) * TL::E_BYTES);
    unrolled<TL::TMW>([&](auto ii) { ex[decltype(ii)::value] = lds_read4_at<decltype(ii)::value * 128>(ea); });
  };
  auto take_exp = [&](int st, uint32_t w) {  // after lds_wait()
#pragma unroll
    for (int i = 0; i < TL::TMW; ++i) {
      asm volatile("" : "+v"(ex[i]));
      sx[i] = ex[i] >> (8 * (st & 3));
    }
    asm volatile("" : "+s"(w));  // the scalar load is waited for here, not where it is issued
    swb = w >> (8 * static_cast<int>(wexp_idx(st) & 3));
  };

  // The accumulators are named here, so the products above stay above (the
  // compiler would otherwise sink them past the barrier to their next use).
  auto pin_acc = [&]() {
#pragma unroll
    for (int i = 0; i < TL::TMW; ++i)
#pragma unroll
      for (int j = 0; j < TL::TNW; ++j) asm volatile("" : "+a"(acc[i][j]));
  };

  if (st1 > st0) {
    // Every stage of the loop issues the same DMA instructions, so that the waits
    // count them exactly; those past the range read nothing and write zeros.
#pragma unroll
    for (int u = 0; u < TL::NS; ++u) issue_all(st0 + u, u);
    wait_vmcnt<(TL::NS - 1) * TL::L>();
    __builtin_amdgcn_s_barrier();
    Frag f0, f1;
    using H0 = std::integral_constant<int, 0>;
    using H1 = std::integral_constant<int, 1>;
    unrolled<NR>([&](auto nn) { read1(f0, 0u, H0{}, nn); });
    read_exp(st0);
    const uint32_t w0 = wexp_load(st0);
    lds_wait();
    tie_all(f0);
    take_exp(st0, w0);

    int slot = 0;
    for (int st = st0; st < st1; ++st) {
      const uint32_t so = static_cast<uint32_t>(slot * TL::STAGE_BYTES);
      const int nslot = slot + 1 == TL::NS ? 0 : slot + 1;
      const uint32_t sn = static_cast<uint32_t>(nslot * TL::STAGE_BYTES);
      const int stn = st + 1 < st1 ? st + 1 : st;
      const uint32_t wn1 = wexp_load(stn);
      // first half stage's products; the second half's fragments come in
      constexpr int RA = (NR + NM - 1) / NM;  // reads after each matrix instruction
      unrolled<NM>([&](auto mm) {
        constexpr int m = decltype(mm)::value;
        mfma1(f0, m / TL::TNW, m % TL::TNW);
        unrolled<RA>([&](auto rr) {
          constexpr int n = m * RA + decltype(rr)::value;
          if constexpr (n < NR) read1(f1, so, H1{}, std::integral_constant<int, n>{});
        });
        __builtin_amdgcn_sched_barrier(0);
      });
      pin_acc();
      lds_wait();
      tie_all(f1);
      // this wave is done with the stage's slot; when all are, and the next
      // stage's loads have landed, the slot takes stage st + NS
      wait_vmcnt<(TL::NS - 2) * TL::L>();
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      if (((st + TL::NS) & 3) == 0) issue_exp(st + TL::NS);
      read_exp(stn);
      constexpr int DA = (TL::L + NM - 1) / NM;  // DMA instructions after each matrix instruction
      unrolled<NM>([&](auto mm) {
        constexpr int m = decltype(mm)::value;
        mfma1(f1, m / TL::TNW, m % TL::TNW);
        unrolled<RA>([&](auto rr) {
          constexpr int n = m * RA + decltype(rr)::value;
          if constexpr (n < NR) read1(f0, sn, H0{}, std::integral_constant<int, n>{});
        });
        unrolled<DA>([&](auto dd) {
          constexpr int k = m * DA + decltype(dd)::value;
          if constexpr (k < TL::L) issue1(st + TL::NS, slot, std::integral_constant<int, k>{});
        });
        __builtin_amdgcn_sched_barrier(0);
      });
      lds_wait();
      tie_all(f0);
      take_exp(stn, wn1);
      slot = nslot;
    }
    wait_vmcnt<0>();  // the DMA past the range is done before the workgroup's LDS is given up
  }

  // lane coordinates taken anew, so that nothing but the accumulators and the
  // loop's own values is live across the loop
  int el = static_cast<int>(threadIdx.x) & 63;
  asm volatile("" : "+v"(el));
  const int erow32 = el & 31, ehalf = el >> 5;
  if (a.nSplit > 1) {
    // this split's fp32 tile, 16 bytes a lane, in the order the join reads it
    f32x4* p = reinterpret_cast<f32x4*>(a.part) +
               ((static_cast<int64_t>(sp) * tiles + (static_cast<int64_t>(rb) * a.nTiles + nt)) * TL::NW + wave) *
                   (TL::TMW * TL::TNW * 256) + el;
#pragma unroll
    for (int i = 0; i < TL::TMW; ++i)
#pragma unroll
      for (int j = 0; j < TL::TNW; ++j) {
        asm volatile("" : "+a"(acc[i][j]));  // one tile at a time leaves the accumulator registers
#pragma unroll
        for (int q = 0; q < 4; ++q)
          p[((i * TL::TNW + j) * 4 + q) * 64] = f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                                                      acc[i][j][4 * q + 3]};
      }
    return;
  }
#pragma unroll
  for (int i = 0; i < TL::TMW; ++i)
#pragma unroll
    for (int j = 0; j < TL::TNW; ++j) {
      asm volatile("" : "+a"(acc[i][j]));
      store_tile<DT>(a, m0 + (wm * TL::TMW + i) * 32 + erow32, n0 + (wn * TL::TNW + j) * 32, acc[i][j], ehalf);
    }
}

// One wave a matrix tile of the output: its splits' sums added in order.
template <int DT, class TL>
__global__ __launch_bounds__(256) void q8_gemm_join(GemmArgs a) {
  const int lane = threadIdx.x & 63;
  constexpr int PT = TL::NW * TL::TMW * TL::TNW;  // matrix tiles of a workgroup tile
  const int64_t tiles = static_cast<int64_t>(a.nRB) * a.nTiles;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (w >= tiles * PT) return;
  const int64_t tile = w / PT;
  const int sub = static_cast<int>(w % PT);
  const int wave = sub / (TL::TMW * TL::TNW), ij = sub % (TL::TMW * TL::TNW);
  const f32x4* p = reinterpret_cast<const f32x4*>(a.part) + (tile * PT + sub) * 256 + lane;
  f32x4 s[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) s[q] = p[q * 64];
  for (int k = 1; k < a.nSplit; ++k) {
    const f32x4* pk = p + static_cast<int64_t>(k) * tiles * PT * 256;
#pragma unroll
    for (int q = 0; q < 4; ++q) s[q] += pk[q * 64];
  }
  f32x16 acc;
#pragma unroll
  for (int q = 0; q < 16; ++q) acc[q] = s[q / 4][q % 4];
  const int64_t m0 = tile / a.nTiles * TL::BM, n0 = tile % a.nTiles * TL::BN;
  const int i = ij / TL::TNW, j = ij % TL::TNW, wm = wave / TL::WN, wn = wave % TL::WN;
  store_tile<DT>(a, m0 + (wm * TL::TMW + i) * 32 + (lane & 31), n0 + (wn * TL::TNW + j) * 32, acc, lane >> 5);
}

// Few rows (T <= 16 TM).  A workgroup owns 16 NJ output columns; its eight
// waves take the stages in turn and their sums meet in LDS.  The weight goes
// from global memory straight into fragments, each row's 128 bytes of a stage
// by two 16-byte loads of four lanes; x stays in the caches.  Lane group g of
// 16 holds chunks g and g + 4 of a stage on both sides.
constexpr int kFewWaves = 8, kFewU = 4;

template <int DT, int TM, int NJ>
__global__ __launch_bounds__(64 * kFewWaves, 2) void q8_gemm_few(GemmArgs a) {
  using T16 = typename Dt<DT>::T;
  __shared__ f32x4 red[kFewWaves][NJ * TM][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, g = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * (16 * NJ);
  const uint8_t* xr[TM];
  const uint8_t* er[TM];
#pragma unroll
  for (int i = 0; i < TM; ++i) {  // rows past T repeat the last one; their sums are not stored
    const int64_t t = min(static_cast<int64_t>(i * 16 + l16), a.T - 1);
    xr[i] = a.xq + t * a.xp + g * 16;
    er[i] = a.xe + t * a.xep;
  }
  const uint8_t* wr[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) wr[j] = a.wq + min(n0 + j * 16 + l16, a.wrows - 1) * a.wp + g * 16;
  const uint8_t* we = a.we + n0 / kQ8Block * a.wep;  // 16 NJ divides 128: one block
  f32x4 acc[NJ][TM];
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int i = 0; i < TM; ++i) acc[j][i] = f32x4{};

  for (int s0 = wave; s0 < a.S; s0 += kFewWaves * kFewU) {
    u32x4 w[kFewU][NJ][2], x[kFewU][TM][2];
    uint32_t ew[kFewU], ex[kFewU][TM];
#pragma unroll
    for (int u = 0; u < kFewU; ++u) {
      const int st = min(s0 + u * kFewWaves, a.S - 1);
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          w[u][j][c] = *reinterpret_cast<const u32x4*>(wr[j] + static_cast<int64_t>(st) * kQ8Block + c * 64);
      ew[u] = we[st];
#pragma unroll
      for (int i = 0; i < TM; ++i) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
          x[u][i][c] = *reinterpret_cast<const u32x4*>(xr[i] + static_cast<int64_t>(st) * kQ8Block + c * 64);
        ex[u][i] = er[i][st];
      }
    }
#pragma unroll
    for (int u = 0; u < kFewU; ++u) {
      if (s0 + u * kFewWaves >= a.S) break;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          auto v8 = [](const u32x4 (&c)[2]) {
            return v8i{static_cast<int>(c[0][0]), static_cast<int>(c[0][1]), static_cast<int>(c[0][2]),
                       static_cast<int>(c[0][3]), static_cast<int>(c[1][0]), static_cast<int>(c[1][1]),
                       static_cast<int>(c[1][2]), static_cast<int>(c[1][3])};
          };
          acc[j][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              v8(w[u][j]), v8(x[u][i]), acc[j][i], 0, 0, 0, static_cast<int>(ew[u]), 0, static_cast<int>(ex[u][i]));
        }
    }
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int i = 0; i < TM; ++i) red[wave][j * TM + i][lane] = acc[j][i];
  __syncthreads();
  // matrix tile k = wave, wave + 8, ..: register q of lane l is output column
  // 4*(l/16) + q of row l%16
  for (int k = wave; k < NJ * TM; k += kFewWaves) {
    f32x4 s = red[0][k][lane];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) s += red[w][k][lane];
    const int64_t t = (k % TM) * 16 + l16, c = n0 + (k / TM) * 16 + 4 * g;
    if (t >= a.T) continue;
    typedef T16 t4 __attribute__((ext_vector_type(4)));
    const t4 o = {Dt<DT>::from_f(s[0]), Dt<DT>::from_f(s[1]), Dt<DT>::from_f(s[2]), Dt<DT>::from_f(s[3])};
    T16* y = static_cast<T16*>(a.y) + t * a.N + c;
    if (a.vec) {  // N % 8 == 0
      if (c < a.N) *reinterpret_cast<t4*>(y) = o;
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (c + q < a.N) y[q] = o[q];
    }
  }
}

#ifndef Q8_BIG_MIN
#define Q8_BIG_MIN 192
#endif
template <bool TRANS>
using BigTile = Q8Tile<2, 2, 4, 4, 2, TRANS>;  // 256 x 256
template <bool TRANS>
using MidTile = Q8Tile<2, 2, 2, 2, 4, TRANS>;  // 128 x 128

constexpr int64_t kFewRows = 64;

struct GemmPlan {
  enum Path { kFew, kBig, kMid } path = kBig;
  int64_t N = 0;
  int S = 0, nSplit = 1;
  int64_t nRB = 0, nTiles = 0;
  int64_t grid = 0;
  size_t bytes = 0;
};

GemmPlan gemm_plan(int64_t T, int64_t out, int64_t in, bool trans) {
  GemmPlan p;
  p.N = trans ? in : out;
  p.S = static_cast<int>(q8_ceil(trans ? out : in, kQ8Block));
  if (!trans && T <= kFewRows) {
    p.path = GemmPlan::kFew;
    p.grid = q8_ceil(p.N, T <= 16 ? 16 : 32);
    return p;
  }
  const int64_t big = q8_ceil(T, 256) * q8_ceil(p.N, 256);
  p.path = big >= Q8_BIG_MIN ? GemmPlan::kBig : GemmPlan::kMid;
  const int64_t b = p.path == GemmPlan::kBig ? 256 : 128;
  p.nRB = q8_ceil(T, b);
  p.nTiles = q8_ceil(p.N, b);
  const int64_t tiles = p.nRB * p.nTiles;
  if (p.path == GemmPlan::kMid) {
    // one workgroup a CU: split the contraction while CUs are idle, at least
    // eight stages a split
    int64_t split = std::min<int64_t>(256 / std::max<int64_t>(tiles, 1), p.S / 8);
    p.nSplit = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(split, 16)));
  }
  p.grid = q8_ceil(tiles * p.nSplit, 8) * 8;
  if (p.nSplit > 1) p.bytes = static_cast<size_t>(tiles) * p.nSplit * b * b * 4;
  return p;
}

template <int DT, class TL>
void launch_tile(const GemmArgs& g, const GemmPlan& p, hipStream_t stream) {
  hipLaunchKernelGGL((q8_gemm_tile<DT, TL>), dim3(static_cast<unsigned>(p.grid)), dim3(TL::NT), 0, stream, g);
  if (p.nSplit > 1) {
    const int64_t waves = p.nRB * p.nTiles * TL::NW * TL::TMW * TL::TNW;
    hipLaunchKernelGGL((q8_gemm_join<DT, TL>), dim3(static_cast<unsigned>(q8_ceil(waves, 4))), dim3(256), 0, stream, g);
  }
}

template <int DT>
void launch_few(const GemmArgs& g, const GemmPlan& p, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.grid)), block(64 * kFewWaves);
  if (g.T <= 16)
    hipLaunchKernelGGL((q8_gemm_few<DT, 1, 1>), grid, block, 0, stream, g);
  else if (g.T <= 32)
    hipLaunchKernelGGL((q8_gemm_few<DT, 2, 2>), grid, block, 0, stream, g);
  else
    hipLaunchKernelGGL((q8_gemm_few<DT, 4, 2>), grid, block, 0, stream, g);
}

template <int DT>
void launch_typed(const GemmArgs& g, const GemmPlan& p, bool trans, hipStream_t stream) {
  if (p.path == GemmPlan::kFew)
    launch_few<DT>(g, p, stream);
  else if (p.path == GemmPlan::kBig)
    trans ? launch_tile<DT, BigTile<true>>(g, p, stream) : launch_tile<DT, BigTile<false>>(g, p, stream);
  else
    trans ? launch_tile<DT, MidTile<true>>(g, p, stream) : launch_tile<DT, MidTile<false>>(g, p, stream);
}

}  // namespace

size_t q8_gemm_workspace_bytes(int64_t T, int64_t out, int64_t in, bool trans) {
  return gemm_plan(T, out, in, trans).bytes;
}
int64_t q8_gemm_max_grid(int64_t T, int64_t out, int64_t in, bool trans) { return gemm_plan(T, out, in, trans).grid; }

hipError_t launch_q8_gemm(const Q8GemmArgs& p) {
  const GemmPlan plan = gemm_plan(p.T, p.out, p.in, p.trans);
  const int64_t K = p.trans ? p.out : p.in;
  GemmArgs g{};
  g.xq = static_cast<const uint8_t*>(p.xq);
  g.xe = static_cast<const uint8_t*>(p.xe);
  g.wq = static_cast<const uint8_t*>(p.wq);
  g.we = static_cast<const uint8_t*>(p.we);
  g.T = p.T;
  g.N = plan.N;
  g.xp = q8_row_bytes(K);
  g.wp = q8_row_bytes(p.in);
  g.xep = q8_exp_bytes(K);
  g.wep = q8_exp_bytes(p.in);
  g.wrows = q8_row_bytes(p.out);
  g.S = plan.S;
  g.nRB = static_cast<int>(plan.nRB);
  g.nTiles = static_cast<int>(plan.nTiles);
  g.nSplit = plan.nSplit;
  g.group = 8;
  g.y = p.y;
  g.vec = plan.N % 8 == 0 && (reinterpret_cast<uintptr_t>(p.y) & 15u) == 0;
  g.part = static_cast<float*>(p.ws);
  if (p.dtype == 0)
    launch_typed<0>(g, plan, p.trans, p.stream);
  else
    launch_typed<1>(g, plan, p.trans, p.stream);
  return hipGetLastError();
}

}  // namespace dora
