// Backward from 8-bit checkpoints, for gfx950: the compose's backward with the
// base in 8-bit blocks, and the gradient of A from x in 8-bit blocks.
//
//   d_base = (g - 1) * dy  (g * dy with add_base), in 16 bits or packed again
//   d_B    = g * s * E,   E = dy^T h                       [out x r]
//   d_mag  = (sum_t dy * base + s * sum_k B * E) / n
//   d_A    = d_h^T x = (x^T d_h)^T                         [r x in]
//
// Both are contractions over the tokens, E = X^T Y with X = dy or x and Y = h or
// d_h, in 16-bit matrix instructions with fp32 sums.
//
// Kernels:
//   q8_rows          one pass over X (and the base).  A workgroup owns 128
//                    columns of X, one block of every row, x up to 384 columns
//                    of Y x a slice of the tokens.  Stages of 32 tokens go
//                    global -> LDS by DMA into a ring.  Eight waves each own 64
//                    x 32 TNW of E: a wave reads the fragments of the next half
//                    stage (16 tokens), transposed by the reads, behind the
//                    matrix instructions of this one, and its other work stands
//                    between them too: d_base, its packing and the column sums;
//                    or, for 8-bit X, the conversion of the next stage's panel
//                    to 16 bits, once a value, into LDS.
//
// Measured at 8192^2, bf16, whole calls back to back (r = 384 / 128 / 16): compose,
// packed d_base 112 / 73 / 58 us, 16-bit 117 / 85 / 82 (from a 16-bit base, by
// dora_lora_compose_bwd, 116 / 96 / 92); gradient of A 77 to 82 / 39 / 30; and at
// 10240 x 27648, r = 512: 550, 577 (648), 369.  Under a kernel trace a call takes
// longer (the gradient at r = 384: 85 from its first kernel's start to its second's
// end), and after a read that evicts the caches 133 / 114 / 111, 137 / 117 / 116
// (144 / 132 / 128) and 81 / 47 / 37.  What bounds it: at narrow r the bytes (r = 16
// packed: 256 MiB of dy, base and d_base, 4.6 TB/s); at wide r the panel of Y, 24
// KiB of DMA a stage into each CU for 4 KiB of the 8-bit X: the return path is busy
// 63 % of the gradient's kernel, the matrix cores 28 %.
// Measured and not kept (packed, 16-bit, gradient at r = 384, where the kept form
// took 122 / 127 / 89 and 573 / 580 / 389 in the same session): four waves of 64 x
// 64 TNW, each converting its own fragments of X, 129 / 125 / 87 and 645 / 584 /
// 388 at 10240 x 27648; at r = 128 two workgroups a CU, with twice the token
// slices, 92 / 105 / 45 against 75 / 85 / 40; a start of every workgroup at another
// stage, slower by 5 % and more; the loads spread over both half stages, the same.
//
//   q8_bwd_finalize, q8_grad_a_finalize
//                    the slices added in order, scaled or transposed, rounded;
//   pad_rows         rows that are not multiples of 8 elements (out of dy, r of h,
//                    B and d_h) are copied into the workspace with zeros behind
//                    them first: a copy of the operand costs less than any path
//                    of the kernel without 16-byte loads.
#include <algorithm>
#include <type_traits>

#include "dma_common.hpp"
#include "q8_common.hpp"

namespace dora {

namespace {

inline size_t al256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
inline int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }

// Transposing LDS reads: in each group of 16 lanes a source lane L gives the
// 8-byte address of four columns of row L/4, and result lane i receives the four
// rows of column i.
// All LDS reads here are inline assembly (the compiler would wait for every DMA
// in flight before each); their results are valid after lds_wait*().
template <int OFF>
__device__ inline u32x2 read_tr16(uint32_t addr) {
  u32x2 v;
  asm volatile("ds_read_b64_tr_b16 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "n"(OFF) : "memory");
  return v;
}
template <int OFF>
__device__ inline u32x2 read8(uint32_t addr) {
  u32x2 v;
  asm volatile("ds_read_b64 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "n"(OFF) : "memory");
  return v;
}
template <int OFF>
__device__ inline uint32_t read4(uint32_t addr) {
  uint32_t v;
  asm volatile("ds_read_b32 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "n"(OFF) : "memory");
  return v;
}

// Tile geometry.  LDS image of a stage's 16-bit panels (X = dy, Y): rows of
// tokens, 256-byte groups of 16 chunks, logical 16-byte chunk c of row t in place
// c ^ (4 * (t % 4)): the transposing reads touch 4 consecutive rows and 2 chunks
// of each, and the 8 (row, chunk) pairs then fall in 8 distinct bank groups.  The
// 8-bit panels (the base, or X) are read along their rows and lie plain; an 8-bit X
// is turned into a 16-bit panel of the same image, two of them behind the ring.
template <int TNW_, bool GRAD_>
struct RowsTile {
  static constexpr int TNW = TNW_;
  static constexpr bool GRAD = GRAD_;  // the gradient of A; else the compose's backward
  static constexpr int WM = 2, WN = 4, NW = 8, NT = 512, TMW = 2;
  static constexpr int BM = 128, BN = 32 * TNW * WN, BK = 32;
  static constexpr int XROWB = 2 * BM, YROWB = 2 * BN;
  static constexpr int P_BYTES = BK * XROWB, X_BYTES = GRAD ? P_BYTES / 2 : P_BYTES, Y_BYTES = BK * YROWB, B_BYTES = GRAD ? 0 : BK * BM;
  static constexpr int E_BYTES = 256;  // a dword with the block's exponent per token
  static constexpr int Y_OFF = X_BYTES, B_OFF = Y_OFF + Y_BYTES, E_OFF = B_OFF + B_BYTES;
  static constexpr int SLOT_BYTES = E_OFF + E_BYTES;
  // (an 8-bit panel is four instructions: waves 4 to 7 load what 0 to 3 do, so that
  // every wave issues the same number)
  static constexpr int XQ = 1, YQ = Y_BYTES / 1024 / NW, BQ = GRAD ? 0 : 1;
  static constexpr int L = XQ + YQ + BQ;  // DMA instructions a wave and stage (wave 0: and the exponents)
  // 8-bit X: two 16-bit panels behind the ring, this stage's and the next one's
  static constexpr int NSMAX = (160 * 1024 - (GRAD ? 2 * P_BYTES : 0)) / SLOT_BYTES, NS = NSMAX < 6 ? NSMAX : 6;
  static constexpr int P_OFF = NS * SLOT_BYTES, LDS_BYTES = P_OFF + (GRAD ? 2 * P_BYTES : 0);
  static constexpr int AHEAD = GRAD ? 2 : 1;  // slots that have landed at a stage's middle
  static constexpr int NM = TMW * TNW;  // matrix instructions of a half stage
  static_assert(Y_BYTES % (1024 * NW) == 0 && NS >= 2 + AHEAD && (NS - 2) * (L + 3) < 64, "ring depth and vmcnt range");
  static_assert((32 + WN) * BM * 4 <= LDS_BYTES, "the epilogue's sums fit the ring");
};

__device__ inline int slot16(int c, int t) { return (c & ~15) | ((c ^ (4 * (t & 3))) & 15); }

struct RowsArgs {
  const void *x, *y;         // X = dy (16 bits) or null, Y [T x r] (16 bits, r % 8 == 0)
  const uint8_t *q8, *e8;    // the base, or X: 8-bit blocks
  int64_t T, nx, r;          // nx: columns of X
  int64_t ldx;               // row pitch of dy in elements: nx rounded up to 8, zeros behind
  int64_t qp, ep;            // bytes of a packed row, of its exponents
  int nCB, nTiles, nSplit;
  float* e_part;             // [nSplit][nx][r]
  // the compose's backward
  const void* B;             // [nx x r]
  const float *mag, *norm;
  float s;
  int add_base;
  void* d_base;              // 16 bits, or null
  uint8_t *dq, *de;          // packed, or null
  float* col_part;           // [nSplit][nTiles][nx]
};

template <int DT, class TL>
__global__ __launch_bounds__(TL::NT, 2) void q8_rows(RowsArgs a) {
  using V8 = typename Dt<DT>::V8;
  using T16 = typename Dt<DT>::T;
  __shared__ __attribute__((aligned(1024))) char smem[TL::LDS_BYTES];
  const uint32_t v = static_cast<uint32_t>(xcd_logical_index());
  const uint32_t nCB = static_cast<uint32_t>(a.nCB), nTl = static_cast<uint32_t>(a.nTiles);
  if (v >= nCB * nTl * static_cast<uint32_t>(a.nSplit)) return;
  // consecutive workgroups share a token slice (one slice of Y per XCD's L2)
  const int nt = static_cast<int>(v % nTl), cb = static_cast<int>((v / nTl) % nCB), sp = static_cast<int>(v / (nTl * nCB));
  const int64_t nx = a.nx, r = a.r;
  const int64_t j0 = static_cast<int64_t>(cb) * TL::BM, k0 = static_cast<int64_t>(nt) * TL::BN;
  const int64_t ts = a.T * sp / a.nSplit, rows = a.T * (sp + 1) / a.nSplit - ts;
  const int S = static_cast<int>((rows + TL::BK - 1) / TL::BK);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / TL::WN, wn = wave % TL::WN;
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_char_t*)smem));
  const bool elem = !TL::GRAD && nt == 0;  // the elementwise part is done by the first block of Y's columns

  // Buffer resources over the token slice: rows past it read zero and are not written.
  auto slice = [&](const void* p, int64_t pitch) {
    return __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(p ? static_cast<const char*>(p) + ts * pitch : nullptr), static_cast<short>(0),
        static_cast<int>(p ? rows * pitch : 0), kBufferWord3);
  };
  const __amdgpu_buffer_rsrc_t rx = TL::GRAD ? slice(a.q8, a.qp) : slice(a.x, a.ldx * 2), ry = slice(a.y, r * 2),
                               rb = slice(elem ? a.q8 : nullptr, a.qp), re = slice(a.e8, a.ep);

  // Per-lane DMA offsets (stage 0).  Instruction q of wave w moves 1 KiB block q*NW
  // + w of its panel, lane l writing bytes 16l .. 16l + 15.
  uint32_t xo[TL::XQ], yo[TL::YQ];
  const int t8 = 8 * (wave & 3) + (lane >> 3), c8 = lane & 7;  // an 8-bit panel's row and place
#pragma unroll
  for (int q = 0; q < TL::XQ; ++q) {
    if constexpr (TL::GRAD) {
      xo[q] = static_cast<uint32_t>(t8 * a.qp + j0 + 16 * c8);
    } else {
      const int t = 4 * (q * TL::NW + wave) + (lane >> 4);
      const int64_t col = j0 + 8 * slot16(lane & 15, t);
      xo[q] = col < a.ldx ? static_cast<uint32_t>((t * a.ldx + col) * 2) : kOob;
    }
  }
#pragma unroll
  for (int q = 0; q < TL::YQ; ++q) {
    const int lin = (q * TL::NW + wave) * 64 + lane, t = lin / (TL::BN / 8);
    const int64_t col = k0 + 8 * slot16(lin % (TL::BN / 8), t);
    yo[q] = col < r ? static_cast<uint32_t>((t * r + col) * 2) : kOob;
  }
  const uint32_t bo = static_cast<uint32_t>(t8 * a.qp + j0 + 16 * c8);
  const uint32_t eo = lane < TL::BK ? static_cast<uint32_t>(lane * a.ep) + (static_cast<uint32_t>(cb) & ~3u) : kOob;
  const int eshift = 8 * (cb & 3);
  const uint32_t xstep = static_cast<uint32_t>(TL::BK * (TL::GRAD ? a.qp : a.ldx * 2));
  const uint32_t ystep = static_cast<uint32_t>(TL::BK * r * 2), qstep = static_cast<uint32_t>(TL::BK * a.qp);
  const uint32_t estep = static_cast<uint32_t>(TL::BK * a.ep);
  // (an offset out of range stays there: it is not advanced)
  auto at = [](uint32_t o, uint32_t step, uint32_t st) { return o == kOob ? kOob : o + step * st; };
  auto issue1 = [&](uint32_t st, int slot, auto kk) {
    constexpr int k = decltype(kk)::value;
    char* so = smem + slot * TL::SLOT_BYTES;
    if constexpr (k < TL::XQ)
      dma16(rx, so + (TL::GRAD ? wave & 3 : wave) * 1024, at(xo[k], xstep, st));
    else if constexpr (k < TL::XQ + TL::YQ)
      dma16(ry, so + TL::Y_OFF + ((k - TL::XQ) * TL::NW + wave) * 1024, at(yo[k - TL::XQ], ystep, st));
    else
      dma16(rb, so + TL::B_OFF + (wave & 3) * 1024, bo + qstep * st);
  };
  auto issue_exp = [&](uint32_t st, int slot) {
    if (wave == 0)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(re, (lds_void_t*)(smem + slot * TL::SLOT_BYTES + TL::E_OFF), 4,
                                               at(eo, estep, st), 0, 0, 0);
  };

  // ---- fragment read addresses within a slot.  In a 16-lane group g = l/16, a
  // 16-bit read covers tokens R0 .. R0 + 3 with R0 = 16 step + 8 (g/2) (+ 4 for the
  // second read).  Y (operand A): result lane i gets column 32 j + sigma(16 (g%2) +
  // i), sigma(p) = 16 ((p/4)%2) + 4 (p/8) + p%4, so that accumulator register q of
  // lane l holds Y column 16 (l/32) + q.  X (operand B): column 32 i + l%32.
  const int g = lane >> 4, L16 = lane & 15, half = lane >> 5;
  const int trow = 8 * (g >> 1) + (L16 >> 2);
  auto addr16 = [&](int off, int rowb, int col) {
    const int c = col >> 3;
    return lds0 + static_cast<uint32_t>(off + trow * rowb + slot16(c, trow) * 16 + (col & 7) * 2);
  };
  uint32_t ya[TL::TNW], xa[TL::TMW];
#pragma unroll
  for (int j = 0; j < TL::TNW; ++j)
    ya[j] = addr16(TL::Y_OFF, TL::YROWB,
                   32 * (wn * TL::TNW + j) + 16 * ((L16 & 3) & 1) + 8 * (g & 1) + 4 * ((L16 & 3) >> 1));
#pragma unroll
  for (int i = 0; i < TL::TMW; ++i)
    xa[i] = addr16(TL::GRAD ? TL::P_OFF : 0, TL::XROWB, 32 * (wm * TL::TMW + i) + 16 * (g & 1) + 4 * (L16 & 3));

  f32x16 acc[TL::TMW][TL::TNW];
#pragma unroll
  for (int i = 0; i < TL::TMW; ++i)
#pragma unroll
    for (int j = 0; j < TL::TNW; ++j) acc[i][j] = f32x16{};

  struct Frag {  // a half stage's fragments
    u32x2 y[TL::TNW][2], x[TL::TMW][2];
  };
  constexpr int RX = 2 * TL::TMW, NR = RX + 2 * TL::TNW;  // reads of X, then of Y
  auto read1 = [&](Frag& f, uint32_t xs, uint32_t ys, auto ss, auto nn) {
    constexpr int s = decltype(ss)::value, n = decltype(nn)::value;
    if constexpr (n < RX) {
      constexpr int i = n / 2, c = n % 2;
      f.x[i][c] = read_tr16<(16 * s + 4 * c) * TL::XROWB>(xa[i] + xs);
    } else {
      constexpr int j = (n - RX) / 2, c = (n - RX) % 2;
      f.y[j][c] = read_tr16<(16 * s + 4 * c) * TL::YROWB>(ya[j] + ys);
    }
  };
  auto tie_all = [&](Frag& f) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int j = 0; j < TL::TNW; ++j) tie2(f.y[j][c]);
#pragma unroll
      for (int i = 0; i < TL::TMW; ++i) tie2(f.x[i][c]);
    }
  };
  auto mfma1 = [&](Frag& f, int i, int j) {
    acc[i][j] = Dt<DT>::mfma32(
        __builtin_bit_cast(V8, u32x4{f.y[j][0][0], f.y[j][0][1], f.y[j][1][0], f.y[j][1][1]}),
        __builtin_bit_cast(V8, u32x4{f.x[i][0][0], f.x[i][0][1], f.x[i][1][0], f.x[i][1][1]}), acc[i][j]);
  };
  auto pin_acc = [&]() {
#pragma unroll
    for (int i = 0; i < TL::TMW; ++i)
#pragma unroll
      for (int j = 0; j < TL::TNW; ++j) asm volatile("" : "+a"(acc[i][j]));
  };

  // ---- the elementwise part of the compose's backward: this thread takes chunk
  // ec (8 columns) of token row et of every stage
  const int et = tid >> 4, ec = tid & 15;
  const int64_t ecol = j0 + 8 * ec;
  float gb[8], colsum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    colsum[e] = 0.0f;
    gb[e] = 0.0f;
    if (elem && ecol + e < nx) {
      const float m = a.mag[ecol + e], n = a.norm[ecol + e];
      gb[e] = a.add_base ? m / n : (m - n) / n;
    }
  }
  const __amdgpu_buffer_rsrc_t rdb = slice(elem ? a.d_base : nullptr, nx * 2),
                               rdq = slice(elem ? a.dq : nullptr, a.qp), rde = slice(elem ? a.de : nullptr, a.ep);
  const bool out16 = elem && a.d_base, outq = elem && a.dq, pair = a.ldx == nx;
  const uint32_t ea = lds0 + static_cast<uint32_t>(et * TL::XROWB + slot16(ec, et) * 16);  // 
  const uint32_t ba = lds0 + static_cast<uint32_t>(TL::B_OFF + et * TL::BM + ec * 8);
  const uint32_t xa4 = lds0 + static_cast<uint32_t>(TL::E_OFF + et * 4);
  u32x4 wd;
  u32x2 wb;
  uint32_t we;
  auto elem_read = [&](uint32_t so) {
    wd = lds_read16_at<0>(ea + so);
    wb = read8<0>(ba + so);
    we = read4<0>(xa4 + so);
  };
  auto elem_tie = [&]() {
    tie(wd);
    tie2(wb);
    asm volatile("" : "+v"(we));
  };
  // ---- 8-bit X: this thread turns chunk ec of token row et into 16 bits, a stage
  // before its products: one pass a value instead of one in every wave along Y
  const uint32_t ra = lds0 + static_cast<uint32_t>(et * TL::BM + ec * 8);
  const uint32_t pa = lds0 + static_cast<uint32_t>(TL::P_OFF + et * TL::XROWB + slot16(ec, et) * 16);
  auto conv_read = [&](uint32_t so) {
    wb = read8<0>(ra + so);
    we = read4<0>(xa4 + so);
  };
  auto conv_tie = [&]() {
    tie2(wb);
    asm volatile("" : "+v"(we));
  };
  auto conv = [&](uint32_t ps) {
    const uint32_t byte = (we >> eshift) & 255u;
    float f[8];
    q8_decode8(uint2{wb[0], wb[1]}, q8_scale(byte), f);
    if (__any(byte >= (DT == 0 ? 247u : 135u))) q8_hold<DT>(f);  // rare: 256 * 2^e is past the type
    const u32x4 o = __builtin_bit_cast(u32x4, f32_to_chunk<DT>(f));
    asm volatile("ds_write_b128 %0, %1" ::"v"(pa + ps), "v"(o) : "memory");
  };
  // one of its six pieces, a few instructions each
  float ed[8], eb[8];
  uint32_t ebyte = 127;
  auto elem_piece = [&](uint32_t st, int piece) {
    const uint32_t t = st * TL::BK + static_cast<uint32_t>(et);
    if (piece == 0) {
      q8_decode8(uint2{wb[0], wb[1]}, q8_scale((we >> eshift) & 255u), eb);
    } else if (piece == 1) {
      chunk_to_f32<DT>(__builtin_bit_cast(Chunk, wd), ed);
    } else if (piece == 2) {
#pragma unroll
      for (int e = 0; e < 8; ++e) colsum[e] = __builtin_fmaf(ed[e], eb[e], colsum[e]);
    } else if (piece == 3) {
#pragma unroll
      for (int e = 0; e < 8; ++e) ed[e] *= gb[e];
    } else if (piece == 4) {
      if (outq) ebyte = q8_exp_byte(q8_block_amax(ed));
    } else {
      if (out16) {
        const uint32_t o = (t * static_cast<uint32_t>(nx) + static_cast<uint32_t>(ecol)) * 2;
        if (pair) {
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f32_to_chunk<DT>(ed)), rdb,
                                                 ecol < nx ? o : kOob, 0, 0);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, Dt<DT>::from_f(ed[e])), rdb,
                                                  ecol + e < nx ? o + 2 * e : kOob, 0, 0);
        }
      }
      if (outq) {
        // columns behind nx have dy = 0 and gb = 0: their packed values are zeros
        const uint2 w = q8_encode8(ed, q8_scale(ebyte));
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{w.x, w.y}, rdq,
                                              t * static_cast<uint32_t>(a.qp) + static_cast<uint32_t>(ecol), 0, 0);
        // the block's byte by lane 0, the exponent row's padding by the last block's other lanes
        const bool pad = cb == a.nCB - 1 && cb + ec < a.ep;
        __builtin_amdgcn_raw_buffer_store_b8(
            static_cast<uint8_t>(ec == 0 ? ebyte : 127u), rde,
            ec == 0 || pad ? t * static_cast<uint32_t>(a.ep) + static_cast<uint32_t>(cb + ec) : kOob, 0, 0);
      }
    }
  };
  // The slot after stage st's has landed when at most what was issued after its
  // loads is outstanding: the loads of NS - 2 stages, and the stores of as many
  // (none is counted before there are so many; more stores than counted, as single
  // 16-bit ones, only make the wait longer).
  const int nstore = (out16 ? 1 : 0) + (outq ? 2 : 0);
  auto wait_next = [&](int st) {
    constexpr int M = TL::NS - 1 - TL::AHEAD, W = M * TL::L;
    const int n = st < M ? 0 : nstore;
    if (n == 0)
      wait_vmcnt<W>();
    else if (n == 1)
      wait_vmcnt<W + M>();
    else if (n == 2)
      wait_vmcnt<W + 2 * M>();
    else
      wait_vmcnt<W + 3 * M>();
  };

  using H0 = std::integral_constant<int, 0>;
  using H1 = std::integral_constant<int, 1>;
  constexpr int RA = (NR + TL::NM - 1) / TL::NM * 2, DA = (TL::L + TL::NM - 1) / TL::NM;
  constexpr int PA = (6 + TL::NM - 1) / TL::NM;  // elementwise pieces behind each instruction

  // Half a stage: the products of `cur` while the fragments `nxt` come in (half s
  // of X at rdx and of Y at rdy).  In the stage's second half its slot loads anew
  // and the elementwise part, read in the first half, is worked on; the first half
  // holds the conversion of the next stage's X, read in the second half before.
  auto half_stage = [&](auto ss, Frag& cur, Frag& nxt, uint32_t rdx, uint32_t rdy, uint32_t st, int wr) {
    constexpr int s = decltype(ss)::value;
    unrolled<TL::NM>([&](auto mm) {
      constexpr int m = decltype(mm)::value;
      mfma1(cur, m / TL::TNW, m % TL::TNW);
      unrolled<RA>([&](auto rr) {
        constexpr int n = m * RA + decltype(rr)::value;
        if constexpr (n < NR) read1(nxt, rdx, rdy, ss, std::integral_constant<int, n>{});
      });
      if constexpr (s == 1 && TL::GRAD && m == 0) conv(((st + 1) & 1) * TL::P_BYTES);
      if constexpr (s == 0) {
        unrolled<DA>([&](auto dd) {
          constexpr int k = m * DA + decltype(dd)::value;
          if constexpr (k < TL::L) issue1(st + TL::NS, wr, std::integral_constant<int, k>{});
        });
        if constexpr (!TL::GRAD) {
          if (elem) {
#pragma unroll
            for (int p = m * PA; p < (m + 1) * PA && p < 6; ++p) elem_piece(st, p);
          }
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    pin_acc();
  };
  auto next = [](int slot) { return slot + 1 == TL::NS ? 0 : slot + 1; };

  if (S > 0) {
#pragma unroll
    for (int u = 0; u < TL::NS; ++u) {  // stages past the slice read zeros
      issue_exp(u, u);
      unrolled<TL::L>([&](auto kk) { issue1(u, u, kk); });
    }
    wait_vmcnt<(TL::NS - TL::AHEAD) * TL::L>();
    __builtin_amdgcn_s_barrier();
    if constexpr (TL::GRAD) {
      conv_read(0u);
      lds_wait();
      conv_tie();
      conv(0u);
      conv_read(static_cast<uint32_t>(TL::SLOT_BYTES));
      lds_wait();
      conv_tie();
      __builtin_amdgcn_s_barrier();
    }
    Frag f0, f1;
    unrolled<NR>([&](auto nn) { read1(f0, 0u, 0u, H0{}, nn); });
    lds_wait();
    tie_all(f0);
    int slot = 0;
    for (int st = 0; st < S; ++st) {
      const int s1 = next(slot);
      const uint32_t so = static_cast<uint32_t>(slot * TL::SLOT_BYTES), so1 = static_cast<uint32_t>(s1 * TL::SLOT_BYTES);
      if constexpr (!TL::GRAD) elem_read(so);
      half_stage(H1{}, f0, f1, TL::GRAD ? (st & 1) * TL::P_BYTES : so, so, static_cast<uint32_t>(st), slot);
      lds_wait();
      tie_all(f1);
      if constexpr (!TL::GRAD) elem_tie();
      wait_next(st);
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      issue_exp(static_cast<uint32_t>(st + TL::NS), slot);
      if constexpr (TL::GRAD) conv_read(static_cast<uint32_t>(next(s1) * TL::SLOT_BYTES));
      half_stage(H0{}, f1, f0, TL::GRAD ? ((st + 1) & 1) * TL::P_BYTES : so1, so1, static_cast<uint32_t>(st), slot);
      lds_wait();
      tie_all(f0);
      if constexpr (TL::GRAD) conv_tie();
      slot = s1;
    }
    wait_vmcnt<0>();
  }
  __syncthreads();

  // ---- epilogue: E's slice, and with it s * sum_k B E and the column sums
  float* red = reinterpret_cast<float*>(smem);  // [32][128] column sums, then [WN][128] sums of B E
  const T16* Bp = static_cast<const T16*>(a.B);
  const int fr = lane & 31;
  float* ep = a.e_part + static_cast<int64_t>(sp) * nx * r;
#pragma unroll
  for (int i = 0; i < TL::TMW; ++i) {
    const int jl = 32 * (wm * TL::TMW + i) + fr;
    const int64_t j = j0 + jl;
    float bsum = 0.0f;
#pragma unroll
    for (int jj = 0; jj < TL::TNW; ++jj) {
      asm volatile("" : "+a"(acc[i][jj]));
      const int64_t k = k0 + 32 * (wn * TL::TNW + jj) + 16 * half;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (j >= nx || k + 8 * c >= r) continue;  // r % 8 == 0: whole chunks
        float* dst = ep + j * r + k + 8 * c;
#pragma unroll
        for (int q = 0; q < 2; ++q)
          *reinterpret_cast<f32x4*>(dst + 4 * q) =
              f32x4{acc[i][jj][8 * c + 4 * q], acc[i][jj][8 * c + 4 * q + 1], acc[i][jj][8 * c + 4 * q + 2],
                    acc[i][jj][8 * c + 4 * q + 3]};
        if constexpr (!TL::GRAD) {
          float bf[8];
          chunk_to_f32<DT>(*reinterpret_cast<const Chunk*>(Bp + j * r + k + 8 * c), bf);
          float u0 = 0.0f, u1 = 0.0f;
#pragma unroll
          for (int q = 0; q < 8; q += 2) {
            u0 = __builtin_fmaf(bf[q], acc[i][jj][8 * c + q], u0);
            u1 = __builtin_fmaf(bf[q + 1], acc[i][jj][8 * c + q + 1], u1);
          }
          bsum += u0 + u1;
        }
      }
    }
    if constexpr (!TL::GRAD) {
      bsum += __shfl_xor(bsum, 32, 64);
      if (half == 0) red[32 * 128 + wn * 128 + jl] = bsum;
    }
  }
  if constexpr (!TL::GRAD) {
#pragma unroll
    for (int e = 0; e < 8; ++e) red[et * 128 + 8 * ec + e] = colsum[e];
    __syncthreads();
    if (tid < TL::BM && j0 + tid < nx) {
      float cs = 0.0f;
      if (elem)
        for (int t = 0; t < 32; ++t) cs += red[t * 128 + tid];
      const float bs = (red[32 * 128 + tid] + red[33 * 128 + tid]) + (red[34 * 128 + tid] + red[35 * 128 + tid]);
      a.col_part[(static_cast<int64_t>(sp) * nTl + nt) * nx + j0 + tid] = cs + a.s * bs;
    }
  }
}

// Rows of n 16-bit elements to rows of np >= n, zeros behind: 8 elements a thread.
__global__ __launch_bounds__(256) void pad_rows(const uint16_t* x, int64_t rows, int64_t n, int64_t np, Chunk* y) {
  const int64_t cpr = np / 8, total = rows * cpr;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < total;
       e += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t t = e / cpr, c = (e - t * cpr) * 8;
    const uint16_t* p = x + t * n;
    Chunk o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = c + 2 * i < n ? p[c + 2 * i] : 0u, hi = c + 2 * i + 1 < n ? p[c + 2 * i + 1] : 0u;
      o.w[i] = lo | hi << 16;
    }
    y[e] = o;
  }
}

void launch_pad(const void* x, int64_t rows, int64_t n, int64_t np, void* y, hipStream_t stream) {
  const int64_t total = rows * (np / 8);
  if (total == 0) return;
  hipLaunchKernelGGL(pad_rows, dim3(static_cast<unsigned>(std::min<int64_t>(q8_ceil(total, 256), 8192))), dim3(256), 0,
                     stream, static_cast<const uint16_t*>(x), rows, n, np, static_cast<Chunk*>(y));
}

// d_mag from the column partials in fp64, and d_B = g * s * (sum of the E slices,
// rows of rp, in order), four elements of a row a thread.
template <int DT>
__global__ __launch_bounds__(256) void q8_bwd_finalize(const float* col_part, int parts, const float* e_part,
                                                       int nSplit, int64_t out, int64_t r, int64_t rp,
                                                       const float* mag, const float* norm, float s, float* d_mag,
                                                       void* d_B) {
  using T16 = typename Dt<DT>::T;
  const int64_t g0 = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t j = g0; j < out; j += stride) {
    double sum = 0.0;
    for (int p = 0; p < parts; ++p) sum += static_cast<double>(col_part[static_cast<int64_t>(p) * out + j]);
    d_mag[j] = static_cast<float>(sum / static_cast<double>(norm[j]));
  }
  if (r == 0) return;
  const int64_t n = out * rp;
  for (int64_t e = g0; e < n / 4; e += stride) {
    const int64_t j = (e * 4) / rp, k = e * 4 - j * rp;
    f32x4 sum = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int p = 0; p < nSplit; ++p) sum += reinterpret_cast<const f32x4*>(e_part + static_cast<int64_t>(p) * n)[e];
    const float gs = (mag[j] / norm[j]) * s;
    T16* o = static_cast<T16*>(d_B) + j * r + k;
    if (r == rp) {
      typedef T16 t4 __attribute__((ext_vector_type(4)));
      *reinterpret_cast<t4*>(o) = t4{Dt<DT>::from_f(gs * sum[0]), Dt<DT>::from_f(gs * sum[1]),
                                     Dt<DT>::from_f(gs * sum[2]), Dt<DT>::from_f(gs * sum[3])};
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (k + q < r) o[q] = Dt<DT>::from_f(gs * sum[q]);
    }
  }
}

// d_A [r x in] = the E slices [in x rp] added in order, transposed through LDS
// in tiles of 64 x 64.
template <int DT>
__global__ __launch_bounds__(256) void q8_grad_a_finalize(const float* e_part, int nSplit, int64_t in, int64_t r,
                                                          int64_t rp, void* d_A) {
  using T16 = typename Dt<DT>::T;
  __shared__ float tile[64][65];
  const int64_t k0 = static_cast<int64_t>(blockIdx.x) * 64, j0 = static_cast<int64_t>(blockIdx.y) * 64;
  const int cx = threadIdx.x & 15, ry = threadIdx.x >> 4;
  const int64_t j = j0 + 4 * cx;  // rp % 8 == 0: the four are inside or outside together
  f32x4 sum[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) sum[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (j < rp) {
    for (int p = 0; p < nSplit; ++p) {
      const float* E = e_part + static_cast<int64_t>(p) * in * rp + j;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t k = min(k0 + ry + 16 * q, in - 1);
        sum[q] += *reinterpret_cast<const f32x4*>(E + k * rp);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) tile[4 * cx + i][ry + 16 * q] = sum[q][i];
  __syncthreads();
  const int kx = threadIdx.x & 63, jy = threadIdx.x >> 6;
  if (k0 + kx >= in) return;
  T16* o = static_cast<T16*>(d_A) + k0 + kx;
  for (int q = jy; q < 64 && j0 + q < r; q += 4) o[(j0 + q) * in] = Dt<DT>::from_f(tile[q][kx]);
}

// Y's columns a workgroup takes, in 128s (least padding, then widest), and token
// slices: one workgroup a CU (it holds most of its LDS), at least eight stages,
// and no slice of any operand (row_bytes: the longest row) of 2 GiB or more.
struct RowsPlan {
  int tn = 1, nCB = 0, nTiles = 0, nSplit = 1;
  size_t off_col = 0, bytes = 0;
};
RowsPlan rows_plan(int64_t T, int64_t nx, int64_t r, int64_t row_bytes) {
  RowsPlan p;
  int64_t best = -1;
  for (int tn = 1; tn <= 3; ++tn) {
    const int64_t pad = q8_ceil(r, 128 * tn) * 128 * tn;
    if (best < 0 || pad <= best) best = pad, p.tn = tn;
  }
  p.nCB = static_cast<int>(q8_ceil(nx, 128));
  p.nTiles = static_cast<int>(q8_ceil(r, 128 * p.tn));
  const int64_t blocks = static_cast<int64_t>(p.nCB) * p.nTiles;
  int64_t split = std::min<int64_t>(q8_ceil(256, blocks), std::max<int64_t>(1, T / 256));
  split = std::max<int64_t>(1, std::min<int64_t>(split, 64));
  p.nSplit = static_cast<int>(std::max(split, q8_ceil(T, INT32_MAX / row_bytes)));
  p.off_col = al256(static_cast<size_t>(p.nSplit) * nx * r * 4);
  p.bytes = p.off_col + static_cast<size_t>(p.nSplit) * p.nTiles * nx * 4;
  return p;
}

struct Q8BwdPlan {
  RowsPlan tile;
  int64_t xp = 0, rp = 0;  // padded row lengths of dy (or d_h's rank) in elements
  size_t off_dy = 0, off_h = 0, off_B = 0, bytes = 0;
  bool pad_x = false, pad_r = false;
};

// nx: columns of X (out, or in); compose: X is dy.
Q8BwdPlan q8_bwd_plan(int64_t T, int64_t nx, int64_t r, bool compose) {
  Q8BwdPlan p;
  p.rp = std::max<int64_t>(8, up8(r));
  p.xp = up8(nx);
  p.pad_x = compose && p.xp != nx;
  p.pad_r = p.rp != r;
  // (a packed row is longer than a 16-bit one below 64 columns)
  p.tile = rows_plan(T, nx, p.rp, std::max({p.xp * 2, p.rp * 2, q8_row_bytes(nx)}));
  size_t at = al256(p.tile.bytes);
  p.off_dy = at;
  if (p.pad_x) at = al256(at + static_cast<size_t>(T) * p.xp * 2);
  p.off_h = at;
  if (p.pad_r) at = al256(at + static_cast<size_t>(T) * p.rp * 2);
  p.off_B = at;
  if (p.pad_r && compose) at = al256(at + static_cast<size_t>(nx) * p.rp * 2);
  p.bytes = at;
  return p;
}

template <bool GRAD>
void launch_rows(const RowsArgs& a, int tn, int dtype, hipStream_t stream) {
  const int64_t total = static_cast<int64_t>(a.nCB) * a.nTiles * a.nSplit;
  const dim3 grid(static_cast<unsigned>(q8_ceil(total, 8) * 8));
  auto go = [&](auto dt, auto t) {
    using TL = RowsTile<decltype(t)::value, GRAD>;
    hipLaunchKernelGGL((q8_rows<decltype(dt)::value, TL>), grid, dim3(TL::NT), 0, stream, a);
  };
  auto by_tile = [&](auto dt) {
    if (tn == 1)
      go(dt, std::integral_constant<int, 1>{});
    else if (tn == 2)
      go(dt, std::integral_constant<int, 2>{});
    else
      go(dt, std::integral_constant<int, 3>{});
  };
  if (dtype == 0)
    by_tile(std::integral_constant<int, 0>{});
  else
    by_tile(std::integral_constant<int, 1>{});
}

}  // namespace

Q8BwdSizes q8_bwd_sizes(int64_t T, int64_t nx, int64_t r, bool compose) {
  const Q8BwdPlan p = q8_bwd_plan(T, nx, r, compose);
  Q8BwdSizes s;
  s.bytes = p.bytes;
  s.grid = std::max<int64_t>(static_cast<int64_t>(p.tile.nCB) * p.tile.nTiles * p.tile.nSplit + 8, q8_ceil(p.rp, 64));
  return s;
}

hipError_t launch_q8_compose_bwd(const Q8ComposeBwdArgs& p) {
  const Q8BwdPlan plan = q8_bwd_plan(p.T, p.out, p.r, true);
  char* ws = static_cast<char*>(p.ws);
  RowsArgs a{};
  a.x = p.dy;
  a.y = p.h;
  a.B = p.B;
  if (plan.pad_x) {
    launch_pad(p.dy, p.T, p.out, plan.xp, ws + plan.off_dy, p.stream);
    a.x = ws + plan.off_dy;
  }
  if (plan.pad_r) {
    launch_pad(p.h, p.T, p.r, plan.rp, ws + plan.off_h, p.stream);
    launch_pad(p.B, p.out, p.r, plan.rp, ws + plan.off_B, p.stream);
    a.y = ws + plan.off_h;
    a.B = ws + plan.off_B;
  }
  a.mag = p.mag;
  a.norm = p.norm;
  a.d_base = p.d_base;
  a.s = p.s;
  a.add_base = p.add_base;
  a.T = p.T;
  a.nx = p.out;
  a.r = plan.rp;
  a.ldx = plan.xp;
  a.nCB = plan.tile.nCB;
  a.nTiles = plan.tile.nTiles;
  a.nSplit = plan.tile.nSplit;
  a.e_part = reinterpret_cast<float*>(ws);
  a.col_part = reinterpret_cast<float*>(ws + plan.tile.off_col);
  a.q8 = static_cast<const uint8_t*>(p.bq);
  a.e8 = static_cast<const uint8_t*>(p.be);
  a.qp = q8_row_bytes(p.out);
  a.ep = q8_exp_bytes(p.out);
  a.dq = static_cast<uint8_t*>(p.dq);
  a.de = static_cast<uint8_t*>(p.de);
  if (p.T > 0) {
    launch_rows<false>(a, plan.tile.tn, p.dtype, p.stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int splits = p.T > 0 ? plan.tile.nSplit : 0, parts = splits * plan.tile.nTiles;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(q8_ceil(std::max(p.out * plan.rp / 4, p.out), 256), 4096)));
  if (p.dtype == 0)
    hipLaunchKernelGGL((q8_bwd_finalize<0>), grid, dim3(256), 0, p.stream, a.col_part, parts, a.e_part, splits, p.out,
                       p.r, plan.rp, p.mag, p.norm, p.s, p.d_mag, p.d_B);
  else
    hipLaunchKernelGGL((q8_bwd_finalize<1>), grid, dim3(256), 0, p.stream, a.col_part, parts, a.e_part, splits, p.out,
                       p.r, plan.rp, p.mag, p.norm, p.s, p.d_mag, p.d_B);
  return hipGetLastError();
}

hipError_t launch_q8_grad_a(const Q8GradAArgs& p) {
  const Q8BwdPlan plan = q8_bwd_plan(p.T, p.in, p.r, false);
  char* ws = static_cast<char*>(p.ws);
  RowsArgs a{};
  a.y = p.dh;
  if (plan.pad_r) {
    launch_pad(p.dh, p.T, p.r, plan.rp, ws + plan.off_h, p.stream);
    a.y = ws + plan.off_h;
  }
  a.T = p.T;
  a.nx = p.in;
  a.r = plan.rp;
  a.ldx = plan.xp;
  a.nCB = plan.tile.nCB;
  a.nTiles = plan.tile.nTiles;
  a.nSplit = plan.tile.nSplit;
  a.e_part = reinterpret_cast<float*>(ws);
  a.q8 = static_cast<const uint8_t*>(p.xq);
  a.e8 = static_cast<const uint8_t*>(p.xe);
  a.qp = q8_row_bytes(p.in);
  a.ep = q8_exp_bytes(p.in);
  if (p.T > 0) {
    launch_rows<true>(a, plan.tile.tn, p.dtype, p.stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int splits = p.T > 0 ? plan.tile.nSplit : 0;
  const dim3 grid(static_cast<unsigned>(q8_ceil(p.in, 64)), static_cast<unsigned>(q8_ceil(p.r, 64)));
  if (p.dtype == 0)
    hipLaunchKernelGGL((q8_grad_a_finalize<0>), grid, dim3(256), 0, p.stream, a.e_part, splits, p.in, p.r, plan.rp,
                       p.d_A);
  else
    hipLaunchKernelGGL((q8_grad_a_finalize<1>), grid, dim3(256), 0, p.stream, a.e_part, splits, p.in, p.r, plan.rp,
                       p.d_A);
  return hipGetLastError();
}

}  // namespace dora
