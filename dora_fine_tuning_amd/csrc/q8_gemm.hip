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
// the price taken for the instruction's rate, twice the 16-bit one's.  Errors
// against 64 bits, of the kernel and of fp32 products: 2.118e-4 and 2.070e-4 (fp16,
// 37 rows of 27648 x 5120), 1.6597e-3 and 1.6591e-3 (bf16, 8192^3).
//
// Kernels:
//   q8_gemm_tile    one workgroup a CU takes tiles of the output, or of the last
//                   tiles ranges of the contraction's stages of 128.  Stages go
//                   global -> LDS by DMA into a ring; fragments are read one
//                   half stage ahead of the matrix instructions that use them,
//                   a few reads behind each instruction, so the matrix pipe is
//                   fed without a pause by one wave per SIMD.  The backward's
//                   weight panel keeps its rows (the contraction axis) and is
//                   transposed by the reads (ds_read_b64_tr_b8);
//   q8_gemm_join    adds the fp32 tiles of a split contraction in order;
//   q8_gemm_few     few rows: the weight is streamed once, straight from global
//                   memory into the fragments of mfma 16x16x128.
//
// What bounds the tiles, at 8192^2 x 8192 with normal values: the card's power.
// The 415 us (2650 TFLOP/s) run at 1.65 to 1.8 GHz with the matrix pipes busy 71%
// of the cycles; the same launch on zeros takes 319 us, at 2.3 GHz.  A stage of the
// 256 x 256 tile takes 2450 cycles, 2048 of them matrix instructions.
#include <algorithm>
#include <type_traits>

#include "dma_common.hpp"
#include "q8_common.hpp"
#include "tile_units.hpp"

namespace dora {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));

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

// Tile geometry: WM x WN waves, each TMW x TNW matrix tiles of 32 x 32 with
// their accumulators in registers; a ring of NS slots of one stage, 128
// contraction steps of both panels.  (Half stages in a ring of twice the slots,
// which load further ahead, fetch half a cache line a row: 8192^2 x 8192 took
// 2880 cycles a stage with them, bound by the L2's requests, 2450 with whole
// lines.)
//
// LDS images of a slot.  X and the forward's W panel: rows of 128 bytes, logical
// 16-byte chunk c of row p in place c ^ ((p/2) % 8): 16 consecutive rows at one
// chunk then fall in 16 distinct bank groups.  The backward's W panel: 128 rows of
// BN bytes; a transposing read touches 8 consecutive rows and two chunks c, c + 1
// (c even), so the chunk is exchanged by the row, leaving its lowest bit alone,
// which spreads the 16 (row, chunk) pairs over the 16 bank groups.
template <int WM_, int WN_, int TMW_, int TNW_, int NS_, bool TRANS_>
struct Q8Tile {
  static constexpr int WM = WM_, WN = WN_, TMW = TMW_, TNW = TNW_, NS = NS_;
  static constexpr bool TRANS = TRANS_;
  static constexpr int NW = WM * WN, NT = 64 * NW;
  static constexpr int BM = 32 * TMW * WM, BN = 32 * TNW * WN, BK = 128;
  static constexpr int X_BYTES = BM * BK, W_BYTES = BN * BK, SLOT_BYTES = X_BYTES + W_BYTES;
  static constexpr int XQ = X_BYTES / 1024 / NW, WQ = W_BYTES / 1024 / NW, L = XQ + WQ;  // DMA instructions a wave
  static constexpr int E_BYTES = BM * 4, NE = 8;  // exponents of the X rows, four stages; slots of them
  static constexpr int LDS_BYTES = NS * SLOT_BYTES + NE * E_BYTES;
  static constexpr int CPR = BN / 16;  // chunks per row of the backward's W panel
  static constexpr int NST = 2 * TMW * TNW;  // 16-byte stores of a wave's tile
  static constexpr int WAIT = (NS - 2) * L;  // DMA instructions younger than the slot waited for
  // a slot's loads stand in the half stage after it is free, or (deeper rings) in
  // that and the next one (8192^2 backward, 65 to 512 rows: 4 to 10 % less; forward
  // 0 to 2 %)
  static constexpr int LA = NS > 2 ? (L + 1) / 2 : L;
  static constexpr int RELAX = NS > 2 ? NS - 2 : NS - 1;  // stages whose slot was loaded before a tile's stores
  static_assert(X_BYTES % (1024 * NW) == 0 && W_BYTES % (1024 * NW) == 0, "whole DMA instructions per wave");
  static_assert(NW % 2 == 0 && BM % 64 == 0 && BM / 64 <= NW, "panel swizzle and exponent DMA");
  static_assert(!TRANS || BN == 128 || BN == 256, "the backward's panel rows");
  static_assert(128 % (32 * TNW) == 0, "a wave's columns lie in one weight block");
  static_assert(NS >= 2 && NS < NE, "an exponent slot outlives the stages in flight");
  static_assert(WAIT + NST < 64, "vmcnt range");
  static_assert(LDS_BYTES <= 160 * 1024, "LDS");
};

struct GemmArgs : TileGrid {
  const uint8_t *xq, *xe, *wq, *we;
  int64_t T, N;      // output rows and columns
  int64_t xp, wp;    // bytes of a row of xq and wq
  int64_t xep, wep;  // bytes of a row of exponents
  int64_t wrows;     // rows of wq (whole tiles)
  void* y;
  int vec;  // 16-byte stores of y
  float* part;
};

// Rows of y from a wave's accumulators: register q of lane l is output column
// 8*(q/4) + 4*(l/32) + q%4 of its tile, row l%32.  Packed in pairs, two groups
// of four columns change places between the lane halves, and each lane then
// holds 8 consecutive columns.  Stores past the matrix are dropped by the buffer
// resource, so that a tile is always the same number of stores.
template <int DT>
__device__ inline void store_tile(__amdgpu_buffer_rsrc_t ry, int vec, uint32_t row, int64_t N, int64_t c0,
                                  const f32x16& acc, int half) {
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
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const uint32_t c = static_cast<uint32_t>(c0) + 16 * g + 8 * half, n = static_cast<uint32_t>(N);
    const uint32_t at = (row * n + c) * 2;
    const u32x4 w = u32x4{p[4 * g], p[4 * g + 1], p[4 * g + 2], p[4 * g + 3]};
    if (vec) {
      __builtin_amdgcn_raw_buffer_store_b128(w, ry, c < n ? at : kOob, 0, 0);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1))), ry,
                                              c + i < n ? at + 2 * i : kOob, 0, 0);
    }
  }
}

// Rows [m, m + most) of y, as far as they exist.
__device__ inline __amdgpu_buffer_rsrc_t rows_of_y(const GemmArgs& a, int64_t m, int most) {
  const int64_t rows = min(max(a.T - m, int64_t(0)), static_cast<int64_t>(most));
  return buffer_of(static_cast<char*>(a.y) + (rows > 0 ? m * a.N * 2 : 0), rows * a.N * 2);
}

// One workgroup a CU, each taking its units in turn.  The ring runs on from one
// unit to the next: while a unit's last slots are worked on, the next one's
// first ones load, and its stores are under way while the next one's products
// run.  Splitting the tiles that do not fill a round of all CUs takes 27648 x 5120
// with 10240 rows backward (800 tiles, 3.1 rounds) from 1340 us to 1160 us.
template <int DT, class TL>
__global__ __launch_bounds__(TL::NT, 1) void q8_gemm_tile(GemmArgs a) {
  __shared__ __attribute__((aligned(1024))) char smem[TL::LDS_BYTES];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / TL::WN, wn = wave % TL::WN;
  const int frow = lane & 31, half = lane >> 5;
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_char_t*)smem));

  Unit cu;
  if (!unit_of(0, a, cu)) return;

  // ---- the issuing side: its unit, and that unit's buffer resources (rows past
  // the operand read zero; past the last unit everything does, so that every half
  // stage issues the same instructions and the waits count them exactly)
  const int xr = wave * 8 + (lane >> 3);  // X rows (and the forward's W rows) of DMA instruction 0
  const uint32_t kc = static_cast<uint32_t>(((lane & 7) ^ ((xr >> 1) & 7)) * 16);
  const uint32_t xo = static_cast<uint32_t>(xr * a.xp) + kc;
  const uint32_t xstep = static_cast<uint32_t>(TL::NW * 8 * a.xp);
  const uint32_t eo = static_cast<uint32_t>((wave * 64 + lane) * a.xep);
  constexpr int RPI = TL::TRANS ? 64 / TL::CPR : 8;  // W rows per DMA instruction
  static_assert((TL::NW * RPI) % 8 == 0, "swizzle period");
  const int tr = wave * RPI + lane / TL::CPR;  // backward: W row of instruction 0, and its logical chunk
  const int tc = (lane % TL::CPR) ^ (TL::CPR == 16 ? 2 * (tr & 7) : 2 * ((tr >> 1) & 3));
  uint32_t wo = static_cast<uint32_t>(xr * a.wp) + kc;
  uint32_t wstep = static_cast<uint32_t>(TL::NW * RPI * a.wp);

  int ik = 0, ist = 0, iend = 0, ig = 0;
  bool live = true;
  __amdgpu_buffer_rsrc_t rx, re, rw;
  const uint8_t* iw = a.wq;
  int64_t in0 = 0;
  // backward: the stage's 128 rows from column n0 on; the last byte that exists
  // is the last row's last, n0 bytes before the end of 128 rows from here
  auto issue_rows = [&]() {
    if constexpr (TL::TRANS)
      rw = buffer_of(iw + (live ? static_cast<int64_t>(ist) * TL::BK * a.wp : 0), live ? TL::BK * a.wp - in0 : 0);
  };
  auto issue_unit = [&](Unit u) {
    ist = u.st0;
    iend = u.st1;
    const int64_t m0 = static_cast<int64_t>(u.rb) * TL::BM, n0 = static_cast<int64_t>(u.nt) * TL::BN;
    const int64_t xrows = live ? min(a.T - m0, static_cast<int64_t>(TL::BM)) : 0;
    rx = buffer_of(a.xq + m0 * a.xp, xrows * a.xp);
    re = buffer_of(a.xe + m0 * a.xep, xrows * a.xep);
    if constexpr (TL::TRANS) {
      iw = a.wq + n0;
      in0 = n0;
      const bool ok = n0 + 16 * tc < a.wp;
      wo = ok ? static_cast<uint32_t>(tr * a.wp + 16 * tc) : kOob;
      wstep = ok ? static_cast<uint32_t>(TL::NW * RPI * a.wp) : 0u;
    } else {
      rw = buffer_of(a.wq + n0 * a.wp, live ? min(a.wrows - n0, static_cast<int64_t>(TL::BN)) * a.wp : 0);
    }
  };
  // DMA instruction k of the issuing side's stage (k compile time)
  auto issue1 = [&](int slot, auto kk) {
    constexpr int k = decltype(kk)::value;
    char* so = smem + slot * TL::SLOT_BYTES;
    const uint32_t at = static_cast<uint32_t>(ist) * TL::BK;
    if constexpr (k < TL::XQ) {
      dma16(rx, so + (k * TL::NW + wave) * 1024, xo + k * xstep + at);
    } else {
      constexpr int q = k - TL::XQ;
      char* d = so + TL::X_BYTES + (q * TL::NW + wave) * 1024;
      if constexpr (TL::TRANS)
        dma16(rw, d, wo + q * wstep);
      else
        dma16(rw, d, wo + q * wstep + at);
    }
  };
  // exponents of the X rows, a dword (four stages) a row, with the first stage
  // of the unit and of every four
  auto issue_exp = [&](bool first) {
    if (!first && (ist & 3) != 0) return;
    ig = (ig + 1) & (TL::NE - 1);
    if (TL::BM / 64 > wave) {
      char* d = smem + TL::NS * TL::SLOT_BYTES + ig * TL::E_BYTES + wave * 256;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(re, (lds_void_t*)d, 4, eo + (ist & ~3), 0, 0, 0);
    }
  };
  bool ifirst = true;
  auto issue_next = [&]() {  // to the next stage, or the next unit's first
    ifirst = false;
    if (++ist == iend) {
      Unit u;
      live = unit_of(++ik, a, u);
      if (!live) u = Unit{0, 0, 0, 1 << 30, 0, -1};
      issue_unit(u);
      ifirst = true;
    }
    issue_rows();
  };
  using H0 = std::integral_constant<int, 0>;
  using H1 = std::integral_constant<int, 1>;

  // ---- fragment read addresses within a slot: half stage s, lane half h takes
  // contraction steps 64s + 32h .. + 31.  (The instruction's own order of the
  // steps within a lane does not matter: both operands use the same.)
  const int sw = (frow >> 1) & 7;
  uint32_t xa[2][2], wa[2][2];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint32_t co = static_cast<uint32_t>(((4 * s + 2 * half + c) ^ sw) * 16);
      xa[s][c] = lds0 + static_cast<uint32_t>((wm * TL::TMW * 32 + frow) * TL::BK) + co;
      wa[s][c] = lds0 + static_cast<uint32_t>(TL::X_BYTES + (wn * TL::TNW * 32 + frow) * TL::BK) + co;
    }
  const uint32_t erow = lds0 + static_cast<uint32_t>(TL::NS * TL::SLOT_BYTES + (wm * TL::TMW * 32 + frow) * 4);
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
  // A half stage's fragments: X rows as two 16-byte reads, W as two (forward)
  // or four transposing reads.
  struct Frag {
    u32x4 x[TL::TMW][2];
    u32x4 w[TL::TRANS ? 1 : TL::TNW][2];
    u32x2 t[TL::TRANS ? TL::TNW : 1][4];
  };
  constexpr int NR = 2 * TL::TMW + (TL::TRANS ? 4 : 2) * TL::TNW;  // reads of a half stage
  auto read1 = [&](Frag& f, uint32_t so, auto ss, auto nn) {
    constexpr int s = decltype(ss)::value, n = decltype(nn)::value;
    if constexpr (n < 2 * TL::TMW) {
      constexpr int i = n / 2, c = n % 2;
      f.x[i][c] = lds_read16_at<i * 32 * TL::BK>(xa[s][c] + so);
    } else if constexpr (!TL::TRANS) {
      constexpr int j = (n - 2 * TL::TMW) / 2, c = n % 2;
      f.w[j][c] = lds_read16_at<j * 32 * TL::BK>(wa[s][c] + so);
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

  // ---- exponents of the computing side.  The weight block's byte by a scalar
  // load: the address is the wave's own and nothing writes there while the kernel
  // runs.  (Columns past the weight have zero panels: any exponent.)
  typedef const uint32_t __attribute__((address_space(4))) const_u32;
  const int nblk = static_cast<int>((TL::TRANS ? a.wp : a.wrows) / kQ8Block);
  const int wep = static_cast<int>(a.wep);  // a weight has below 2^30 blocks
  auto wexp_idx = [&](const Unit& u) -> int {
    const int wb = min((u.nt * TL::BN + wn * TL::TNW * 32) / static_cast<int>(kQ8Block), nblk - 1);
    return TL::TRANS ? u.st0 * wep + wb : wb * wep + u.st0;
  };
  const int wexp_step = TL::TRANS ? wep : 1;
  auto wexp_load = [&](int idx) -> uint32_t {
    return ((const_u32*)(reinterpret_cast<uintptr_t>(a.we)))[idx >> 2];
  };
  uint32_t ex[TL::TMW];
  int cg = 0;  // exponent slot of the computing side
  auto read_exp = [&]() {
    const uint32_t ea = erow + static_cast<uint32_t>(cg * TL::E_BYTES);
    unrolled<TL::TMW>([&](auto ii) { ex[decltype(ii)::value] = lds_read4_at<decltype(ii)::value * 128>(ea); });
  };
  auto take_exp = [&](int st, uint32_t w, int idx) {  // after lds_wait()
#pragma unroll
    for (int i = 0; i < TL::TMW; ++i) {
      asm volatile("" : "+v"(ex[i]));
      sx[i] = ex[i] >> (8 * (st & 3));
    }
    asm volatile("" : "+s"(w));  // the scalar load is waited for here, not where it is issued
    swb = w >> (8 * (idx & 3));
  };
  // The accumulators are named here, so the products above stay above (the
  // compiler would otherwise sink them past the barrier to their next use).
  auto pin_acc = [&]() {
#pragma unroll
    for (int i = 0; i < TL::TMW; ++i)
#pragma unroll
      for (int j = 0; j < TL::TNW; ++j) asm volatile("" : "+a"(acc[i][j]));
  };

  // An accumulator is cleared by a short product of zeros, which takes its zero
  // addend as an inline constant (a zero vector would need registers that the
  // accumulators occupy).
  auto clear = [&](int i, int j) {
    uint32_t z = 0;
    asm volatile("" : "+v"(z));
    const bf16x8 zv = __builtin_bit_cast(bf16x8, u32x4{z, z, z, z});
    acc[i][j] = Dt<0>::mfma32(zv, zv, f32x16{});
    asm volatile("" : "+a"(acc[i][j]));
  };

  // ---- fill the ring
  issue_unit(cu);
  issue_rows();
#pragma unroll
  for (int s = 0; s < TL::NS; ++s) {
    issue_exp(ifirst);
    constexpr int all = TL::L, part = TL::LA;
    if (s + 1 < TL::NS || part == all) {
      unrolled<all>([&](auto kk) { issue1(s, kk); });
      issue_next();
    } else {
      unrolled<part>([&](auto kk) { issue1(s, kk); });
    }
  }
  wait_vmcnt<(TL::NS - 2) * TL::L + TL::LA>();
  __builtin_amdgcn_s_barrier();
  Frag f0, f1;
  cg = 1;
  unrolled<NR>([&](auto nn) { read1(f0, 0u, H0{}, nn); });
  read_exp();
  int widx = wexp_idx(cu);
  {
    const uint32_t w = wexp_load(widx);
    lds_wait();
    tie_all(f0);
    take_exp(cu.st0, w, widx);
  }

  // the unit worked on, and what comes after it
  int st = cu.st0, ck = 0, nst0 = 0;
  int nwidx = 0;
  bool more = false;
  auto look_ahead = [&]() {
    Unit n;
    more = unit_of(ck + 1, a, n);
    nst0 = more ? n.st0 : cu.st0;  // past the last unit: anything readable
    nwidx = more ? wexp_idx(n) : widx;
  };
  look_ahead();
#pragma unroll
  for (int i = 0; i < TL::TMW; ++i)
#pragma unroll
    for (int j = 0; j < TL::TNW; ++j) clear(i, j);

  // Half a stage: the products of fragments `cur`, while fragments `nxt` come in
  // (half s of the slot at rd).  Both reads and DMA instructions stand behind the
  // first matrix instructions, RA and DA a piece, so that the last ones cover
  // their latency.
  int slot = 0;
  int relax = 0;  // stages until the last tile's stores must be done
  constexpr int RA = 2 * ((NR + NM - 1) / NM);
  auto half_stage = [&](auto ss, Frag& cur, Frag& nxt, uint32_t rd, int wr) {
    unrolled<NM>([&](auto mm) {
      constexpr int m = decltype(mm)::value;
      mfma1(cur, m / TL::TNW, m % TL::TNW);
      unrolled<RA>([&](auto rr) {
        constexpr int n = m * RA + decltype(rr)::value;
        if constexpr (n < NR) read1(nxt, rd, ss, std::integral_constant<int, n>{});
      });
      // the stage's second half: its slot begins to load anew; first half: the rest
      constexpr int k0 = decltype(ss)::value == 0 ? 0 : TL::LA, k1 = decltype(ss)::value == 0 ? TL::LA : TL::L;
      constexpr int DA = (k1 - k0 + NM - 1) / NM;
      unrolled<DA>([&](auto dd) {
        constexpr int k = k0 + m * DA + decltype(dd)::value;
        if constexpr (k < k1) issue1(wr, std::integral_constant<int, k>{});
      });
      __builtin_amdgcn_sched_barrier(0);
    });
    pin_acc();
  };

  while (true) {
    const int s1 = slot + 1 == TL::NS ? 0 : slot + 1;
    const uint32_t rd0 = static_cast<uint32_t>(slot * TL::SLOT_BYTES), rd1 = static_cast<uint32_t>(s1 * TL::SLOT_BYTES);
    // the next stage: this unit's, or the next unit's first
    const bool last = st + 1 == cu.st1;
    const int nst = last ? nst0 : st + 1;
    widx = last ? nwidx : widx + wexp_step;
    const uint32_t wn1 = wexp_load(widx);

    half_stage(H1{}, f0, f1, rd0, slot == 0 ? TL::NS - 1 : slot - 1);
    if constexpr (TL::LA < TL::L) issue_next();
    lds_wait();
    tie_all(f1);
    // this wave has read the slot; the next slot has landed; when that holds for
    // all waves, the slot takes the issuing side's next stage
    if (relax > 0) {
      --relax;
      wait_vmcnt<TL::WAIT + TL::NST>();
    } else {
      wait_vmcnt<TL::WAIT>();
    }
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    issue_exp(ifirst);
    if (last || (nst & 3) == 0) cg = (cg + 1) & (TL::NE - 1);
    read_exp();
    half_stage(H0{}, f1, f0, rd1, slot);
    if constexpr (TL::LA == TL::L) issue_next();
    lds_wait();
    tie_all(f0);
    if (last) {
      // lane coordinates taken anew, so that nothing but the accumulators and the
      // loop's own values is live across the loop
      int el = static_cast<int>(threadIdx.x) & 63;
      asm volatile("" : "+v"(el));
      const uint32_t er = static_cast<uint32_t>(el & 31);
      const int eh = el >> 5;
      const bool part = cu.tail >= 0 && a.nSplit > 1;
      // a split's fp32 tile: 16 bytes a lane, in the order the join reads it
      f32x4* p = reinterpret_cast<f32x4*>(a.part) +
                 ((static_cast<int64_t>(cu.split) * (a.nRB * a.nTiles - a.whole) + cu.tail) * TL::NW + wave) *
                     (TL::TMW * TL::TNW * 256) + el;
      const __amdgpu_buffer_rsrc_t ry =
          rows_of_y(a, static_cast<int64_t>(cu.rb) * TL::BM + wm * TL::TMW * 32, TL::TMW * 32);
      const int64_t c0 = static_cast<int64_t>(cu.nt) * TL::BN + wn * TL::TNW * 32;
#pragma unroll
      for (int i = 0; i < TL::TMW; ++i)
#pragma unroll
        for (int j = 0; j < TL::TNW; ++j) {
          asm volatile("" : "+a"(acc[i][j]));  // one tile at a time leaves the accumulator registers
          if (part) {
            if (static_cast<int64_t>(cu.rb) * TL::BM + (wm * TL::TMW + i) * 32 < a.T)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                p[((i * TL::TNW + j) * 4 + q) * 64] = f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1],
                                                            acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          } else {
            store_tile<DT>(ry, a.vec, i * 32 + er, a.N, c0 + j * 32, acc[i][j], eh);
          }
          clear(i, j);
        }
      if (!part && a.vec)
        relax = TL::RELAX;
      else
        wait_vmcnt<0>();
      if (!more) break;
      ++ck;
      unit_of(ck, a, cu);
      look_ahead();
    }
    take_exp(nst, wn1, widx);
    st = nst;
    slot = s1;
  }
  wait_vmcnt<0>();  // the DMA past the last unit is done before the workgroup's LDS is given up
}

// One wave a matrix tile of the output: its splits' sums added in order.
template <int DT, class TL>
__global__ __launch_bounds__(256) void q8_gemm_join(GemmArgs a) {
  const int lane = threadIdx.x & 63;
  constexpr int PT = TL::NW * TL::TMW * TL::TNW;  // matrix tiles of a workgroup tile
  const int64_t ntail = static_cast<int64_t>(a.nRB) * a.nTiles - a.whole;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (w >= ntail * PT) return;
  const int64_t tail = w / PT;
  const int sub = static_cast<int>(w % PT);
  const int wave = sub / (TL::TMW * TL::TNW), ij = sub % (TL::TMW * TL::TNW);
  int rb, nt;
  tile_of(static_cast<uint32_t>(a.whole + tail), a, rb, nt);
  const int i = ij / TL::TNW, j = ij % TL::TNW, wm = wave / TL::WN, wn = wave % TL::WN;
  const int64_t m = static_cast<int64_t>(rb) * TL::BM + (wm * TL::TMW + i) * 32;
  if (m >= a.T) return;  // rows past the last: not written either
  const f32x4* p = reinterpret_cast<const f32x4*>(a.part) + (tail * PT + sub) * 256 + lane;
  f32x4 s[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) s[q] = p[q * 64];
  for (int k = 1; k < a.nSplit; ++k) {
    const f32x4* pk = p + static_cast<int64_t>(k) * ntail * PT * 256;
#pragma unroll
    for (int q = 0; q < 4; ++q) s[q] += pk[q * 64];
  }
  f32x16 acc;
#pragma unroll
  for (int q = 0; q < 16; ++q) acc[q] = s[q / 4][q % 4];
  store_tile<DT>(rows_of_y(a, m, 32), a.vec, static_cast<uint32_t>(lane & 31), a.N,
                 static_cast<int64_t>(nt) * TL::BN + (wn * TL::TNW + j) * 32, acc, lane >> 5);
}

// Few rows (T <= 8; the rows of one 16-row matrix tile).  A workgroup owns 16 output columns; its 16 waves take the
// stages in turn and their sums meet in LDS.  The weight goes from global memory
// straight into fragments of mfma 16x16x128, each row's 128 bytes of a stage by
// two 16-byte loads of four lanes, four stages in flight a wave; the rows stay in
// the caches.  Lane group g of 16 holds chunks g and g + 4 of a stage on both
// sides.  Bound by HBM: 5.5 TB/s of weight at 27648 x 5120 with one row.  Eight
// waves were 0 to 5% slower, 32 columns a workgroup 10 to 25% (one row).
constexpr int kFewWaves = 16, kFewU = 4;

template <int DT>
__global__ __launch_bounds__(64 * kFewWaves) void q8_gemm_few(GemmArgs a) {
  using T16 = typename Dt<DT>::T;
  __shared__ f32x4 red[kFewWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, g = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  // rows past T repeat the last one; their sums are not stored
  const int64_t t = min(static_cast<int64_t>(l16), a.T - 1);
  const uint8_t* xr = a.xq + t * a.xp + g * 16;
  const uint8_t* er = a.xe + t * a.xep;
  const uint8_t* wr = a.wq + min(n0 + l16, a.wrows - 1) * a.wp + g * 16;
  const uint8_t* we = a.we + n0 / kQ8Block * a.wep;  // 16 divides 128: one block
  f32x4 acc = f32x4{};
  for (int s0 = wave; s0 < a.S; s0 += kFewWaves * kFewU) {
    u32x4 w[kFewU][2], x[kFewU][2];
    uint32_t ew[kFewU], ex[kFewU];
#pragma unroll
    for (int u = 0; u < kFewU; ++u) {
      const int64_t st = min(s0 + u * kFewWaves, a.S - 1);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        w[u][c] = *reinterpret_cast<const u32x4*>(wr + st * kQ8Block + c * 64);
        x[u][c] = *reinterpret_cast<const u32x4*>(xr + st * kQ8Block + c * 64);
      }
      ew[u] = we[st];
      ex[u] = er[st];
    }
#pragma unroll
    for (int u = 0; u < kFewU; ++u) {
      if (s0 + u * kFewWaves >= a.S) break;
      auto v8 = [](const u32x4 (&c)[2]) {
        return v8i{static_cast<int>(c[0][0]), static_cast<int>(c[0][1]), static_cast<int>(c[0][2]),
                   static_cast<int>(c[0][3]), static_cast<int>(c[1][0]), static_cast<int>(c[1][1]),
                   static_cast<int>(c[1][2]), static_cast<int>(c[1][3])};
      };
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v8(w[u]), v8(x[u]), acc, 0, 0, 0,
                                                             static_cast<int>(ew[u]), 0, static_cast<int>(ex[u]));
    }
  }
  red[wave][lane] = acc;
  __syncthreads();
  // register q of lane l is output column 4*(l/16) + q of row l%16
  if (wave > 0) return;
  f32x4 s = red[0][lane];
#pragma unroll
  for (int w = 1; w < kFewWaves; ++w) s += red[w][lane];
  const int64_t c = n0 + 4 * g;
  if (l16 >= a.T) return;
  typedef T16 t4 __attribute__((ext_vector_type(4)));
  const t4 o = {Dt<DT>::from_f(s[0]), Dt<DT>::from_f(s[1]), Dt<DT>::from_f(s[2]), Dt<DT>::from_f(s[3])};
  T16* y = static_cast<T16*>(a.y) + static_cast<int64_t>(l16) * a.N + c;
  if (a.vec) {  // N % 8 == 0
    if (c < a.N) *reinterpret_cast<t4*>(y) = o;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (c + q < a.N) y[q] = o[q];
  }
}

// An empty contraction: zeros (the kernels above need at least one stage).
__global__ __launch_bounds__(256) void q8_gemm_zero(uint16_t* y, int64_t n) {
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < n;
       e += static_cast<int64_t>(gridDim.x) * 256)
    y[e] = 0;
}

template <bool TRANS>
using BigTile = Q8Tile<2, 2, 4, 4, 2, TRANS>;  // 256 x 256
template <bool TRANS>
using TallTile = Q8Tile<2, 2, 4, 2, 3, TRANS>;  // 256 x 128
template <bool TRANS>
using HighTile = Q8Tile<2, 2, 3, 2, 3, TRANS>;  // 192 x 128
template <bool TRANS>
using MidTile = Q8Tile<2, 2, 2, 2, 4, TRANS>;  // 128 x 128
template <bool TRANS>
using LowTile = Q8Tile<1, 4, 2, 1, 6, TRANS>;  // 64 x 128, a deep ring: the weight's stream
// forward alone (64 columns of the backward's weight rows are half cache lines)
using SlimTile = Q8Tile<2, 2, 3, 1, 4, false>;   // 192 x 64
using SmallTile = Q8Tile<2, 2, 1, 1, 7, false>;  // 64 x 64

// Up to here the weight's stream decides and every wave reads the rows for
// itself; beyond, 16 rows a wave cost as much as its 16 columns, and tiles of 64
// rows share them.  27648 x 5120, us: 26 with 1 row; 42 with 16 rows here, 31 in
// tiles.  8192^2: 16 with 1 row, 19 with 8, 22 with 16, 21.5 in tiles.
constexpr int64_t kFewRows = 8;

struct GemmPlan {
  enum Path { kSmall, kSlim, kLow, kMid, kHigh, kTall, kBig, kFew } path = kBig;
  int64_t N = 0;
  int S = 0, nSplit = 1;
  int64_t nRB = 0, nTiles = 0, whole = 0;
  int64_t grid = 0;
  size_t bytes = 0;
};

// Tiles of bm x bn: as many rounds of one whole tile a CU as there are, and the
// rest in up to 16 ranges of stages each (at least four stages), whichever number
// is expected to be fastest.  Returns the expected microseconds: a stage of the
// tile (13 % more where the reads transpose), 1.4 for the start and end of a
// unit, and for a split 3.0 + 0.43 a range for the join's launch and sums and
// 0.25 a MB of fp32 partials, written and read.
double split_plan(GemmPlan& p, int64_t T, int64_t bm, int64_t bn, double stage_us) {
  p.nRB = q8_ceil(T, bm);
  p.nTiles = q8_ceil(p.N, bn);
  const int64_t tiles = p.nRB * p.nTiles;
  const int64_t rounds = tiles / kCUs, rest = tiles - rounds * kCUs;
  p.whole = rounds * kCUs;
  p.nSplit = 1;
  const double unit_us = 1.4;
  double best = 0.0;
  if (rest > 0) {
    best = p.S * stage_us + unit_us;
    // a tile's rows that exist are written, on the mean of the tiles
    const double mb = static_cast<double>(rest) * bn * 4e-6 * static_cast<double>(T) / static_cast<double>(p.nRB);
    for (int s = 2; s <= 16 && p.S / s >= 4; ++s) {
      const double c =
          static_cast<double>(q8_ceil(rest * s, kCUs)) * (static_cast<double>(q8_ceil(p.S, s)) * stage_us + unit_us) +
          3.0 + 0.43 * s + 0.25 * mb * s;
      if (c < best) best = c, p.nSplit = s;
    }
  }
  p.grid = std::min<int64_t>(kCUs, q8_ceil(p.whole + rest * p.nSplit, 8) * 8);
  p.bytes = p.nSplit > 1 ? static_cast<size_t>(rest) * p.nSplit * bm * bn * 4 : 0;
  return static_cast<double>(rounds) * (p.S * stage_us + unit_us) + best;
}

// The tile is the one expected to be fastest.  The times are fitted to 5257 calls
// (six weights from 1024 x 8192 to 27648 x 5120, both directions, 9 to 8192 rows,
// every tile, 1 to 16 ranges); over them the plan's call takes 0.8 % more than the
// fastest measured one on the mean, 12 % at most.  Tiles of 64 rows for up to 64
// rows and of 128 and 256 beyond took 4.8 %, 37 % at most.  us, the chosen tile and
// those: 27648 x 5120 with 256 rows 48 / 64, 8192^2 with 300 rows 32 / 37, 4096^2
// with 256 rows 15 / 19.  (These are calls of the product back to back; under a
// kernel trace the one of 32 takes 36.)
GemmPlan gemm_plan(int64_t T, int64_t out, int64_t in, bool trans) {
  GemmPlan p;
  p.N = trans ? in : out;
  p.S = static_cast<int>(q8_ceil(trans ? out : in, kQ8Block));
  if (!trans && T <= kFewRows) {
    p.path = GemmPlan::kFew;
    p.grid = q8_ceil(p.N, 16);
    return p;
  }
  static constexpr struct {
    GemmPlan::Path path;
    int64_t bm, bn;
    double us;
  } tiles[] = {{GemmPlan::kSmall, 64, 64, 0.31},
               {GemmPlan::kSlim, 192, 64, 0.46},
               {GemmPlan::kLow, 64, 128, 0.41},
               {GemmPlan::kMid, 128, 128, 0.55},
               {GemmPlan::kHigh, 192, 128, 0.69},
               {GemmPlan::kTall, 256, 128, 0.85},
               {GemmPlan::kBig, 256, 256, 1.40}};
  GemmPlan best;
  double least = 0.0;
  for (const auto& t : tiles) {
    if (trans && t.bn < 128) continue;
    GemmPlan q = p;
    q.path = t.path;
    const double us = split_plan(q, T, t.bm, t.bn, trans ? 1.13 * t.us : t.us);
    if (least == 0.0 || us < least) least = us, best = q;
  }
  return best;
}

template <int DT, class TL>
void launch_tile(const GemmArgs& g, const GemmPlan& p, hipStream_t stream) {
  hipLaunchKernelGGL((q8_gemm_tile<DT, TL>), dim3(static_cast<unsigned>(p.grid)), dim3(TL::NT), 0, stream, g);
  if (p.nSplit > 1) {
    const int64_t waves = (p.nRB * p.nTiles - p.whole) * TL::NW * TL::TMW * TL::TNW;
    hipLaunchKernelGGL((q8_gemm_join<DT, TL>), dim3(static_cast<unsigned>(q8_ceil(waves, 4))), dim3(256), 0, stream, g);
  }
}

template <int DT>
void launch_few(const GemmArgs& g, const GemmPlan& p, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.grid)), block(64 * kFewWaves);
  hipLaunchKernelGGL((q8_gemm_few<DT>), grid, block, 0, stream, g);
}

template <int DT>
void launch_typed(const GemmArgs& g, const GemmPlan& p, bool trans, hipStream_t stream) {
  switch (p.path) {
    case GemmPlan::kFew:
      return launch_few<DT>(g, p, stream);
    case GemmPlan::kSmall:
      return launch_tile<DT, SmallTile>(g, p, stream);
    case GemmPlan::kSlim:
      return launch_tile<DT, SlimTile>(g, p, stream);
    case GemmPlan::kLow:
      return trans ? launch_tile<DT, LowTile<true>>(g, p, stream) : launch_tile<DT, LowTile<false>>(g, p, stream);
    case GemmPlan::kMid:
      return trans ? launch_tile<DT, MidTile<true>>(g, p, stream) : launch_tile<DT, MidTile<false>>(g, p, stream);
    case GemmPlan::kHigh:
      return trans ? launch_tile<DT, HighTile<true>>(g, p, stream) : launch_tile<DT, HighTile<false>>(g, p, stream);
    case GemmPlan::kTall:
      return trans ? launch_tile<DT, TallTile<true>>(g, p, stream) : launch_tile<DT, TallTile<false>>(g, p, stream);
    case GemmPlan::kBig:
      return trans ? launch_tile<DT, BigTile<true>>(g, p, stream) : launch_tile<DT, BigTile<false>>(g, p, stream);
  }
}

}  // namespace

size_t q8_gemm_workspace_bytes(int64_t T, int64_t out, int64_t in, bool trans) {
  return gemm_plan(T, out, in, trans).bytes;
}
int64_t q8_gemm_max_grid(int64_t T, int64_t out, int64_t in, bool trans) {
  const GemmPlan p = gemm_plan(T, out, in, trans);
  return std::max(p.grid, p.nRB * p.nTiles * 16);  // units of work (tiles in up to 16 ranges) are numbered in 32 bits
}

hipError_t launch_q8_gemm(const Q8GemmArgs& p) {
  const GemmPlan plan = gemm_plan(p.T, p.out, p.in, p.trans);
  const int64_t K = p.trans ? p.out : p.in;
  if (K == 0) {
    const int64_t n = p.T * plan.N;
    hipLaunchKernelGGL(q8_gemm_zero, dim3(static_cast<unsigned>(std::min<int64_t>(q8_ceil(n, 256), 4096))), dim3(256),
                       0, p.stream, static_cast<uint16_t*>(p.y), n);
    return hipGetLastError();
  }
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
  g.whole = static_cast<int>(plan.whole);
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
