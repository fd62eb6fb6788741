// The tile kernel of the row (token) contractions E = X^T Y, shared by the
// 16-bit backward (lora_bwd.hip) and the one that works from 8-bit blocks
// (q8_bwd.hip): tile geometry, kernel, launch plan.
#pragma once

#include <algorithm>
#include <type_traits>

#include "dma_common.hpp"
#include "dora_common.hpp"
#include "lora_compose_kernels.hpp"
#include "q8_common.hpp"

namespace dora {

namespace {

__host__ __device__ inline int64_t bcdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Transposing LDS read: in each group of 16 lanes, source lane L gives an
// 8-byte address (4 consecutive 16-bit elements of one row); result lane i
// receives element i%4 of the source lanes i/4, i/4 + 4, i/4 + 8, i/4 + 12.
// With source lane L addressing row R0 + L/4 at column F(L%4), lane i gets the
// 4 elements of column F(i/4) + i%4 in rows R0 .. R0 + 3.
// Issued as inline assembly, like the other fragment reads (the builtin would
// make the compiler wait for every DMA in flight before each read); the result
// is valid after lds_wait() / lds_wait_keep(), and tie2() orders its uses after
// that wait.
__device__ inline u32x2 lds_read_tr(uint32_t addr) {
  u32x2 v;
  asm volatile("ds_read_b64_tr_b16 %0, %1" : "=v"(v) : "v"(addr) : "memory");
  return v;
}
__device__ inline void tie2(u32x2& v) { asm volatile("" : "+v"(v)); }
__device__ inline u32x2 lds_read8(uint32_t addr) {
  u32x2 v;
  asm volatile("ds_read_b64 %0, %1" : "=v"(v) : "v"(addr) : "memory");
  return v;
}
__device__ inline uint32_t lds_read4(uint32_t addr) {
  uint32_t v;
  asm volatile("ds_read_b32 %0, %1" : "=v"(v) : "v"(addr) : "memory");
  return v;
}
// As the reads, so that the compiler does not wait for every DMA in flight first.
__device__ inline void lds_write16(uint32_t addr, u32x4 v) {
  asm volatile("ds_write_b128 %0, %1" ::"v"(addr), "v"(v) : "memory");
}

// Tile: 128 output columns (X, 32*TM with TM = 4, WM = 2 waves along them) x
// 128*TN rank columns (Y, WN = 4 waves along them); a wave owns TMW = 2 x TN
// tiles of 32x32.  A K stage is 32 tokens: the X panel holds 32 dy rows of 128
// columns (256 bytes), the Y panel 32 h rows of 128*TN rank columns.  Within
// each 16-chunk (256-byte) group of a row, logical 16-byte chunk c of row t sits
// in slot c ^ (4 * (t % 4)): the transposing reads touch 4 consecutive rows and
// 2 chunks per row, and the 8 (row, chunk) pairs then fall in 8 distinct bank
// groups.
// BASE adds the third panel, the base rows of the X panel's tokens and
// columns, laid out like the X panel; the plain contraction has none.
// Roles: NW = 8 tile waves read fragments, run MFMAs and (with BASE) do the
// stage's elementwise part; NDMA = 4 DMA waves (one per SIMD) only issue the
// ring's loads, so the tile waves never stall on the texture path that takes
// a stage's loads.  Every vector-memory instruction of a DMA wave's stage
// loop is a DMA of the ring, which keeps the stage waits exact.
// DUAL (plain contraction only): the Y rows hold two column blocks that add
// into the same output, Y[t][c] and Y[t][ny + c] (the hi and lo halves of a
// value carried as a pair); a stage then holds both Y panels and every
// accumulator takes one MFMA from each, so X is streamed once for both.
// KIND 1 (with BASE): the base panel comes in 8-bit blocks, 128 bytes a token
// row, exactly one block of the row; its exponent byte is loaded by the tile
// waves a stage ahead, and d_base may leave packed the same way.
// KIND 2 (plain contraction): X comes in 8-bit blocks.  A DMA wave turns the
// 1 KiB it has itself loaded (8 token rows) into the 16-bit X panel of the
// stage, in one of two buffers beside the ring, while the tile waves work on
// the other; converting there costs each value one pass instead of one in each
// of the four waves along Y.
enum BwdKind { kBwd16 = 0, kBwdBase8 = 1, kBwdX8 = 2 };
template <int TN_, int NS_, bool BASE_, bool DUAL_ = false, int KIND_ = kBwd16>
struct BwdTile {
  static constexpr int TN = TN_, NS = NS_, KIND = KIND_;
  static constexpr bool BASE = BASE_, DUAL = DUAL_, BASE8 = KIND == kBwdBase8, X8 = KIND == kBwdX8;
  static constexpr int NYP = DUAL ? 2 : 1;  // Y panels per stage
  static constexpr int WM = 2, WN = 4, NW = 8, NDMA = 4, NT = 64 * (NW + NDMA), TM = 4, TMW = 2;
  static constexpr int BM = 128, BN = 128 * TN, BK = 32;
  static constexpr int XROWB = BM * 2, YROWB = BN * 2;  // bytes per token row
  static constexpr int X_BYTES = BK * XROWB, Y_BYTES = BK * YROWB;
  static constexpr int B_BYTES = !BASE ? 0 : BASE8 ? X_BYTES / 2 : X_BYTES;
  // the ring's X panel; in 8 bits: the values, then a dword with the block's exponent per DMA lane
  static constexpr int RX_BYTES = X8 ? X_BYTES / 2 + 4 * 64 * NDMA : X_BYTES;
  static constexpr int B_OFF = RX_BYTES + NYP * Y_BYTES, STAGE_BYTES = RX_BYTES + NYP * Y_BYTES + B_BYTES;
  static constexpr int XI = X_BYTES / 1024, YI = Y_BYTES / 1024;  // 1 KiB DMA blocks per stage and panel
  static constexpr int XQ = XI / NDMA, YQ = YI / NDMA;  // per DMA wave
  static constexpr int L = (X8 ? 2 : XQ) + NYP * YQ + (!BASE ? 0 : BASE8 ? XQ / 2 : XQ);
  static constexpr int XBUF = NS * STAGE_BYTES;  // 8-bit X: the two converted panels
  static constexpr int GB = NS * STAGE_BYTES;  // 8-bit base: the columns' factor of d_base, fp32
  static constexpr int LDS_BYTES = NS * STAGE_BYTES + (X8 ? 2 * X_BYTES : 0) + (BASE8 ? 4 * BM : 0);
  // the widest tile with the elementwise part reads one K step's fragments at
  // a time: both steps' would not fit the registers of three waves per SIMD
  static constexpr bool ONE_STEP = (BASE && TN == 3) || DUAL;
  static_assert(KIND == kBwd16 || (BASE8 ? BASE : !BASE && !DUAL), "8-bit base with the base panel, 8-bit X without");
  static_assert(KIND == kBwd16 || XQ == 2, "one DMA instruction a wave for an 8-bit panel");
  static_assert(!(BASE && DUAL), "the dual Y panels are for the plain contraction");
  static_assert(XI % NDMA == 0 && YI % NDMA == 0, "panels split into whole DMA groups per DMA wave");
  static_assert(NW * 64 == BK * 16, "one 16-byte chunk of a stage's dy and base rows per tile-wave thread");
  static_assert(LDS_BYTES <= 160 * 1024, "LDS");
  static_assert(NS >= 2 && (NS - 2) * L < 64, "ring depth and vmcnt range");
  static_assert(ONE_STEP || 2 * (TMW + TN) < 16, "one K step's fragment reads within the lgkmcnt range");
};

// slot of logical 16-byte chunk c in token row t (see BwdTile)
__device__ inline int bwd_slot(int c, int t) { return (c & ~15) | ((c ^ (4 * (t & 3))) & 15); }

struct BwdArgs {
  const void *dy, *base, *h, *B;
  const float *mag, *norm;
  void* d_base;
  float s;
  int add_base;
  int64_t T, out, r;
  int64_t ldx;  // row pitch of dy in elements: out, or out rounded up to 8 (KIND 1, zeros behind out)
  int64_t ldy;  // row pitch of h (and h2) in elements: r, or 2r with DUAL panels
  int nCB, nTiles, nSplit;
  float* e_part;    // [nSplit][out][r]: the E slices
  float* col_part;  // [nSplit][nTiles][out]: sum_t dy * base (tile 0 only) + s * sum_k B E
  // plain contraction only: the contraction axis continues over the rows of
  // other matrices, dy2 [T2 x out] and h2 [T2 x r]; slice sp takes rows
  // [T2 sp / nSplit, T2 (sp + 1) / nSplit) of them after its own rows of dy, h
  const void *dy2, *h2;
  int64_t T2;
  // 8-bit blocks: the base (KIND 1) or X (KIND 2), bytes per row of values and
  // of exponents; the packed d_base (KIND 1, may be null), same pitches
  const uint8_t *q8, *e8;
  int64_t qp, ep;
  uint8_t *dq8, *de8;
};

// Wait for the current stage's DMA while the younger loads already issued stay
// in flight: n younger stages (at most NS-2) of L loads each.  Younger stores
// (d_base) only make the wait longer.
template <class TL, int N = TL::NS - 2>
__device__ inline void bwd_wait(int n) {
  if constexpr (N == 0) {
    wait_vmcnt<0>();
  } else {
    if (n >= N)
      wait_vmcnt<N * TL::L>();
    else
      bwd_wait<TL, N - 1>(n);
  }
}

template <int DT, class TL>
__global__ __launch_bounds__(TL::NT, 1) void lora_bwd_dma(BwdArgs a) {
  using V8 = typename Dt<DT>::V8;
  using T16 = typename Dt<DT>::T;
  __shared__ __attribute__((aligned(1024))) char smem[TL::LDS_BYTES];

  const uint32_t v = static_cast<uint32_t>(xcd_logical_index());
  const uint32_t nCB = static_cast<uint32_t>(a.nCB), nTl = static_cast<uint32_t>(a.nTiles);
  if (v >= nCB * nTl * static_cast<uint32_t>(a.nSplit)) return;
  // consecutive workgroups share a token slice (one slice of h per XCD's L2)
  const int nt = static_cast<int>(v % nTl);
  const int cb = static_cast<int>((v / nTl) % nCB);
  const int sp = static_cast<int>(v / (nTl * nCB));
  const int64_t T = a.T, out = a.out, r = a.r, ldx = a.ldx, ldy = a.ldy;
  const int64_t j0 = static_cast<int64_t>(cb) * TL::BM, k0 = static_cast<int64_t>(nt) * TL::BN;
  const int64_t ts = T * sp / a.nSplit, te = T * (sp + 1) / a.nSplit;
  // second row segment (plain contraction only; empty when T2 == 0)
  const int64_t ts2 = a.T2 * sp / a.nSplit, te2 = a.T2 * (sp + 1) / a.nSplit;
  const int S1 = static_cast<int>(bcdiv(te - ts, TL::BK));
  const int S = S1 + static_cast<int>(bcdiv(te2 - ts2, TL::BK));
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool dma_wave = wave >= TL::NW;
  const int wm = wave / TL::WN, wn = wave % TL::WN;
  const bool want_base = TL::BASE && nt == 0;  // the elementwise part is done by the first rank block
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_char_t*)smem));
  // epilogue: [32][128] column sums, then [WN][128] rank-block sums
  float* red = reinterpret_cast<float*>(smem);

  if (dma_wave) {
    // ---- DMA waves: the ring's loads, and (with the base panel) the
    // elementwise part of each stage
    const int dw = wave - TL::NW;
    // buffer resources over the token slice; rows past it read zero
    const int64_t rows = te - ts;
    const __amdgpu_buffer_rsrc_t rdy = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(TL::X8 ? nullptr : static_cast<const char*>(a.dy) + ts * ldx * 2), static_cast<short>(0),
        static_cast<int>(TL::X8 ? 0 : rows * ldx * 2), kBufferWord3);
    const __amdgpu_buffer_rsrc_t rbase = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(TL::BASE && !TL::BASE8 ? static_cast<const char*>(a.base) + ts * ldx * 2 : nullptr),
        static_cast<short>(0), static_cast<int>(TL::BASE && !TL::BASE8 ? rows * ldx * 2 : 0), kBufferWord3);
    // 8-bit blocks of the token slice and their exponents
    const __amdgpu_buffer_rsrc_t rq8 = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(TL::KIND ? a.q8 + ts * a.qp : nullptr), static_cast<short>(0),
        static_cast<int>(TL::KIND ? rows * a.qp : 0), kBufferWord3);
    const __amdgpu_buffer_rsrc_t re8 = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(TL::X8 ? a.e8 + ts * a.ep : nullptr), static_cast<short>(0),
        static_cast<int>(TL::X8 ? rows * a.ep : 0), kBufferWord3);
    const __amdgpu_buffer_rsrc_t rh = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(static_cast<const char*>(a.h) + ts * ldy * 2), static_cast<short>(0),
        static_cast<int>(rows * ldy * 2), kBufferWord3);
    const int64_t rows2 = te2 - ts2;
    const __amdgpu_buffer_rsrc_t rdy2 = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(rows2 > 0 ? static_cast<const char*>(a.dy2) + ts2 * ldx * 2 : nullptr),
        static_cast<short>(0), static_cast<int>(rows2 * ldx * 2), kBufferWord3);
    const __amdgpu_buffer_rsrc_t rh2 = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(rows2 > 0 ? static_cast<const char*>(a.h2) + ts2 * ldy * 2 : nullptr),
        static_cast<short>(0), static_cast<int>(rows2 * ldy * 2), kBufferWord3);

    // Per-lane DMA offsets (stage 0).  Instruction q of DMA wave d moves 1 KiB
    // block b = q*NDMA + d of its panel, lane l writing bytes 16l .. 16l + 15.
    // X: a block is 4 dy rows of 256 bytes, so lane l fills slot l%16 of row
    // 4b + l/16 and fetches the logical chunk that slot holds (bwd_slot is its
    // own inverse within a 16-chunk group).  Y: linear 16-byte slot b*64 + l of
    // the 32 x BN panel, row (b*64 + l) / (BN/8).
    uint32_t xo[TL::XQ], yo[TL::YQ];
    bool xok[TL::XQ], yok[TL::YQ];
#pragma unroll
    for (int q = 0; q < TL::XQ; ++q) {
      const int b = q * TL::NDMA + dw;
      const int t = 4 * b + (lane >> 4), sl = lane & 15;
      const int c = bwd_slot(sl, t);
      const int64_t col = j0 + 8 * c;
      xok[q] = col < ldx;
      xo[q] = static_cast<uint32_t>((t * ldx + col) * 2);
    }
#pragma unroll
    for (int q = 0; q < TL::YQ; ++q) {
      const int b = q * TL::NDMA + dw;
      const int lin = b * 64 + lane;
      const int t = lin / (TL::BN / 8), sl = lin % (TL::BN / 8);
      const int c = bwd_slot(sl, t);
      const int64_t col = k0 + 8 * c;
      yok[q] = col < r;
      yo[q] = static_cast<uint32_t>((t * ldy + col) * 2);
    }
    // 8-bit panel: lane l takes 16-byte chunk l%8 of row 8*dw + l/8 of its block
    const int t8 = 8 * dw + (lane >> 3), c8 = lane & 7;
    const uint32_t qo = static_cast<uint32_t>(t8 * a.qp + j0 + 16 * c8), qstep = static_cast<uint32_t>(TL::BK * a.qp);
    const uint32_t blk = static_cast<uint32_t>(cb);  // BM == the block width
    const uint32_t eo = static_cast<uint32_t>(t8 * a.ep) + (blk & ~3u), estep = static_cast<uint32_t>(TL::BK * a.ep);
    const uint32_t xstep = static_cast<uint32_t>(TL::BK * ldx * 2), ystep = static_cast<uint32_t>(TL::BK * ldy * 2);
    // stages [0, S1) read the slice's rows of dy and h, stages [S1, S) those of
    // dy2 and h2 (same row pitches, so the same per-lane offsets); a segment's
    // last stage reads zeros past its rows
    auto issue = [&](int st, int slot) {
      char* so = smem + slot * TL::STAGE_BYTES;
      const bool seg2 = st >= S1;
      const __amdgpu_buffer_rsrc_t rx = seg2 ? rdy2 : rdy, ry = seg2 ? rh2 : rh;
      const uint32_t ss = static_cast<uint32_t>(seg2 ? st - S1 : st);
      if constexpr (TL::X8) {
        dma16(rq8, so + dw * 1024, qo + ss * qstep);
        __builtin_amdgcn_raw_ptr_buffer_load_lds(re8, (lds_void_t*)(so + TL::X_BYTES / 2 + dw * 256), 4,
                                                 eo + ss * estep, 0, 0, 0);
      } else {
#pragma unroll
        for (int q = 0; q < TL::XQ; ++q)
          dma16(rx, so + (q * TL::NDMA + dw) * 1024, xok[q] ? xo[q] + ss * xstep : kOob);
      }
#pragma unroll
      for (int q = 0; q < TL::YQ; ++q)
        dma16(ry, so + TL::RX_BYTES + (q * TL::NDMA + dw) * 1024, yok[q] ? yo[q] + ss * ystep : kOob);
      if constexpr (TL::DUAL) {  // the second Y panel: the same rows, r columns further
#pragma unroll
        for (int q = 0; q < TL::YQ; ++q)
          dma16(ry, so + TL::RX_BYTES + TL::Y_BYTES + (q * TL::NDMA + dw) * 1024,
                yok[q] ? yo[q] + ss * ystep + static_cast<uint32_t>(r * 2) : kOob);
      }
      if constexpr (TL::BASE8) {
        dma16(rq8, so + TL::B_OFF + dw * 1024, want_base ? qo + ss * qstep : kOob);
      } else if constexpr (TL::BASE) {  // never with a second segment
#pragma unroll
        for (int q = 0; q < TL::XQ; ++q)
          dma16(rbase, so + TL::B_OFF + (q * TL::NDMA + dw) * 1024,
                want_base && xok[q] ? xo[q] + ss * xstep : kOob);
      }
    };

    for (int u = 0; u < TL::NS - 1; ++u)
      if (u < S) issue(u, u);
    int slot = 0;
    for (int st = 0; st < S; ++st) {
      bwd_wait<TL>(S - 1 - st);
      if constexpr (TL::X8) {
        // this wave's own block: 16 values a lane, times their row's power of
        // two, to two 16-byte chunks of the X panel (laid out as the DMA's)
        const uint32_t raw = lds0 + static_cast<uint32_t>(slot * TL::STAGE_BYTES);
        u32x4 w = lds_read16(raw + static_cast<uint32_t>(dw * 1024 + lane * 16));
        uint32_t ew = lds_read4(raw + static_cast<uint32_t>(TL::X_BYTES / 2 + dw * 256 + lane * 4));
        lds_wait();
        tie(w);
        asm volatile("" : "+v"(ew));
        const float scale = q8_scale((ew >> (8 * (blk & 3))) & 255u);
        const uint32_t xrow = lds0 + static_cast<uint32_t>(TL::XBUF + (st & 1) * TL::X_BYTES + t8 * TL::XROWB);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float f[8];
          q8_decode8(uint2{w[2 * k], w[2 * k + 1]}, scale, f);
          q8_hold<DT>(f);
          lds_write16(xrow + static_cast<uint32_t>(bwd_slot(2 * c8 + k, t8) * 16),
                      __builtin_bit_cast(u32x4, f32_to_chunk<DT>(f)));
        }
        lds_wait();
      }
      __builtin_amdgcn_s_barrier();
      if (st + TL::NS - 1 < S) issue(st + TL::NS - 1, slot == 0 ? TL::NS - 1 : slot - 1);
      slot = slot == TL::NS - 1 ? 0 : slot + 1;
    }
    // Epilogue.  The ring is free once every wave is past its last read.
    __syncthreads();
  } else {
    // ---- tile waves: fragment reads and MFMAs
    // Fragment read addresses (within a stage slot; add the slot's offset).  In a
    // 16-lane group g = l/16 (i = l%16), a read covers tokens R0 .. R0 + 3 with
    // R0 = 16*step + 8*(g/2) (+ 4 for the second read of a fragment).  Y side
    // (MFMA operand A, rank columns): result lane i must get rank column
    // 32*kt + sigma(16*(g%2) + i), sigma(p) = 16*((p/4)%2) + 4*(p/8) + p%4, so that
    // accumulator register q of lane l holds rank column 16*(l/32) + q; source
    // lane L therefore addresses column 32*kt + 16*((L%4)%2) + 8*(g%2) + 4*((L%4)/2).
    // X side (operand B, output columns): lane i gets column 32*jt + 16*(g%2) + i,
    // so source lane L addresses column 32*jt + 16*(g%2) + 4*(L%4).
    const int g = lane >> 4, L = lane & 15;
    const int rsrc_row = 8 * (g >> 1) + (L >> 2);  // token row within a K step, first read
    auto tr_addr = [&](uint32_t panel, int rowb, int row, int col) {
      const int c = col >> 3;
      return panel + static_cast<uint32_t>(row * rowb + bwd_slot(c, row) * 16 + (col & 7) * 2);
    };
    // per (step, read) the row differs; the column part is per tile
    int ycol[TL::TN], xcol[TL::TMW];
#pragma unroll
    for (int j = 0; j < TL::TN; ++j)
      ycol[j] = 32 * (wn * TL::TN + j) + 16 * ((L & 3) & 1) + 8 * (g & 1) + 4 * ((L & 3) >> 1);
#pragma unroll
    for (int i = 0; i < TL::TMW; ++i) xcol[i] = 32 * (wm * TL::TMW + i) + 16 * (g & 1) + 4 * (L & 3);

    f32x16 acc[TL::TMW][TL::TN];
#pragma unroll
    for (int i = 0; i < TL::TMW; ++i)
#pragma unroll
      for (int j = 0; j < TL::TN; ++j) acc[i][j] = f32x16{};

    // Elementwise part: tile-wave thread tid takes token row tid/16 of each
    // stage and the 8 output columns of chunk tid%16.
    const int et = tid >> 4, ec = tid & 15;
    const int64_t ecol = j0 + 8 * ec;
    const bool eok = want_base && ecol < out;
    float gb[8], colsum[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      colsum[e] = 0.0f;
      gb[e] = 0.0f;
      if (eok && (!TL::BASE8 || ecol + e < out)) {
        const float m = a.mag[ecol + e], n = a.norm[ecol + e];
        gb[e] = a.add_base ? m / n : (m - n) / n;
      }
    }
    T16* dbase = static_cast<T16*>(a.d_base);
    // the widest tile has no registers to keep the factors in beside the packing:
    // with an 8-bit base they wait in LDS (each thread reads back its own write)
    const uint32_t gaddr = lds0 + static_cast<uint32_t>(TL::GB + 32 * ec);
    if constexpr (TL::BASE8) {
      lds_write16(gaddr, __builtin_bit_cast(u32x4, f32x4{gb[0], gb[1], gb[2], gb[3]}));
      lds_write16(gaddr + 16, __builtin_bit_cast(u32x4, f32x4{gb[4], gb[5], gb[6], gb[7]}));
      lds_wait();
    }
    // 8-bit base: this thread's row's exponent byte, loaded a stage ahead
    // (buffer resources over the token slice: 32-bit offsets, and rows past the
    // slice read zero and are not written)
    auto slice = [&](const void* p, int64_t pitch) {
      return __builtin_amdgcn_make_buffer_rsrc(
          const_cast<char*>(TL::BASE8 && p ? static_cast<const char*>(p) + ts * pitch : nullptr),
          static_cast<short>(0), static_cast<int>(TL::BASE8 && p && want_base ? (te - ts) * pitch : 0), kBufferWord3);
    };
    const __amdgpu_buffer_rsrc_t re = slice(a.e8, a.ep), rdb = slice(a.d_base, out * 2), rdq = slice(a.dq8, a.qp),
                                 rde = slice(a.de8, a.ep);
    const uint32_t ep32 = static_cast<uint32_t>(a.ep), qp32 = static_cast<uint32_t>(a.qp);
    const uint32_t out32 = static_cast<uint32_t>(out), j32 = static_cast<uint32_t>(j0);
    auto base_exp = [&](uint32_t t) -> uint32_t {
      return __builtin_amdgcn_raw_buffer_load_b8(re, t * ep32 + static_cast<uint32_t>(cb), 0, 0);
    };
    uint32_t be_next = TL::BASE8 ? base_exp(static_cast<uint32_t>(et)) : 127u;

    int slot = 0;
    for (int st = 0; st < S; ++st) {
      __builtin_amdgcn_s_barrier();  // the DMA waves' loads of stage st have landed
      const uint32_t sp0 = lds0 + static_cast<uint32_t>(slot * TL::STAGE_BYTES);
      const uint32_t xp = TL::X8 ? lds0 + static_cast<uint32_t>(TL::XBUF + (st & 1) * TL::X_BYTES) : sp0;
      const uint32_t yp = sp0 + TL::RX_BYTES;
      const uint32_t be_cur = be_next;
      if constexpr (TL::BASE8) be_next = base_exp(static_cast<uint32_t>((st + 1) * TL::BK + et));
      if constexpr (!TL::ONE_STEP) {
        // both K steps' fragment reads in flight, then each step's MFMAs after its
        // reads have landed (the halves of a fragment are joined after the wait)
        u32x2 xl[2][TL::TMW], xh[2][TL::TMW], yl[2][TL::TN], yh[2][TL::TN];
#pragma unroll
        for (int step = 0; step < 2; ++step) {
          const int row = 16 * step + rsrc_row;
#pragma unroll
          for (int i = 0; i < TL::TMW; ++i) {
            xl[step][i] = lds_read_tr(tr_addr(xp, TL::XROWB, row, xcol[i]));
            xh[step][i] = lds_read_tr(tr_addr(xp, TL::XROWB, row + 4, xcol[i]));
          }
#pragma unroll
          for (int j = 0; j < TL::TN; ++j) {
            yl[step][j] = lds_read_tr(tr_addr(yp, TL::YROWB, row, ycol[j]));
            yh[step][j] = lds_read_tr(tr_addr(yp, TL::YROWB, row + 4, ycol[j]));
          }
        }
#pragma unroll
        for (int step = 0; step < 2; ++step) {
          if (step == 0)
            lds_wait_keep<2 * (TL::TMW + TL::TN)>();
          else
            lds_wait();
          u32x4 fx[TL::TMW], fy[TL::TN];
#pragma unroll
          for (int i = 0; i < TL::TMW; ++i) {
            tie2(xl[step][i]);
            tie2(xh[step][i]);
            fx[i] = u32x4{xl[step][i][0], xl[step][i][1], xh[step][i][0], xh[step][i][1]};
          }
#pragma unroll
          for (int j = 0; j < TL::TN; ++j) {
            tie2(yl[step][j]);
            tie2(yh[step][j]);
            fy[j] = u32x4{yl[step][j][0], yl[step][j][1], yh[step][j][0], yh[step][j][1]};
          }
#pragma unroll
          for (int i = 0; i < TL::TMW; ++i)
#pragma unroll
            for (int j = 0; j < TL::TN; ++j)
              acc[i][j] = Dt<DT>::mfma32(__builtin_bit_cast(V8, fy[j]), __builtin_bit_cast(V8, fx[i]), acc[i][j]);
        }
      } else {
        // one K step's fragments at a time (fewer registers); with DUAL the
        // second Y panel's fragments feed the same accumulators
#pragma unroll
        for (int step = 0; step < 2; ++step) {
          const int row = 16 * step + rsrc_row;
          u32x2 xl[TL::TMW], xh[TL::TMW], yl[TL::NYP][TL::TN], yh[TL::NYP][TL::TN];
#pragma unroll
          for (int i = 0; i < TL::TMW; ++i) {
            xl[i] = lds_read_tr(tr_addr(xp, TL::XROWB, row, xcol[i]));
            xh[i] = lds_read_tr(tr_addr(xp, TL::XROWB, row + 4, xcol[i]));
          }
#pragma unroll
          for (int pn = 0; pn < TL::NYP; ++pn)
#pragma unroll
            for (int j = 0; j < TL::TN; ++j) {
              yl[pn][j] = lds_read_tr(tr_addr(yp + pn * TL::Y_BYTES, TL::YROWB, row, ycol[j]));
              yh[pn][j] = lds_read_tr(tr_addr(yp + pn * TL::Y_BYTES, TL::YROWB, row + 4, ycol[j]));
            }
          lds_wait();
          u32x4 fx[TL::TMW];
#pragma unroll
          for (int i = 0; i < TL::TMW; ++i) {
            tie2(xl[i]);
            tie2(xh[i]);
            fx[i] = u32x4{xl[i][0], xl[i][1], xh[i][0], xh[i][1]};
          }
#pragma unroll
          for (int pn = 0; pn < TL::NYP; ++pn) {
            u32x4 fy[TL::TN];
#pragma unroll
            for (int j = 0; j < TL::TN; ++j) {
              tie2(yl[pn][j]);
              tie2(yh[pn][j]);
              fy[j] = u32x4{yl[pn][j][0], yl[pn][j][1], yh[pn][j][0], yh[pn][j][1]};
            }
#pragma unroll
            for (int i = 0; i < TL::TMW; ++i)
#pragma unroll
              for (int j = 0; j < TL::TN; ++j)
                acc[i][j] = Dt<DT>::mfma32(__builtin_bit_cast(V8, fy[j]), __builtin_bit_cast(V8, fx[i]), acc[i][j]);
          }
        }
      }
      if constexpr (TL::BASE8) {
        if (want_base) {
          const uint32_t t = static_cast<uint32_t>(st * TL::BK + et);
          u32x4 wd = lds_read16(xp + static_cast<uint32_t>(et * TL::XROWB + bwd_slot(ec, et) * 16));
          u32x2 wb = lds_read8(sp0 + static_cast<uint32_t>(TL::B_OFF + et * TL::BM + ec * 8));
          u32x4 ga = lds_read16(gaddr), gc = lds_read16(gaddr + 16);
          lds_wait();
          tie(wd);
          tie2(wb);
          tie(ga);
          tie(gc);
          const f32x4 g0 = __builtin_bit_cast(f32x4, ga), g1 = __builtin_bit_cast(f32x4, gc);
          float dyv[8], bv[8], o[8];
          chunk_to_f32<DT>(__builtin_bit_cast(Chunk, wd), dyv);
          q8_decode8(uint2{wb[0], wb[1]}, q8_scale(be_cur), bv);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            o[e] = (e < 4 ? g0[e & 3] : g1[e & 3]) * dyv[e];
            colsum[e] = __builtin_fmaf(dyv[e], bv[e], colsum[e]);
          }
          if (a.d_base) {
            const uint32_t at = (t * out32 + j32 + 8 * ec) * 2;
            if (ldx == out) {
              __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f32_to_chunk<DT>(o)), rdb,
                                                     ecol < out ? at : kOob, 0, 0);
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, Dt<DT>::from_f(o[e])), rdb,
                                                      ecol + e < out ? at + 2 * e : kOob, 0, 0);
            }
          }
          if (a.dq8) {
            // columns behind out have dy = 0 and gb = 0: their packed values are zeros
            const uint32_t byte = q8_exp_byte(q8_max16(q8_amax8(o)));
            const uint2 w = q8_encode8(o, q8_inv_scale(byte));
            __builtin_amdgcn_raw_buffer_store_b64(u32x2{w.x, w.y}, rdq, t * qp32 + j32 + 8 * ec, 0, 0);
            // the block's byte by lane 0, the exponent row's padding by the last block's other lanes
            const bool pad = cb == a.nCB - 1 && cb + ec < a.ep;
            __builtin_amdgcn_raw_buffer_store_b8(static_cast<uint8_t>(ec == 0 ? byte : 127u), rde,
                                                 ec == 0 || pad ? t * ep32 + static_cast<uint32_t>(cb + ec) : kOob, 0, 0);
          }
        }
      } else if (TL::BASE && eok) {
        const int64_t t = ts + static_cast<int64_t>(st) * TL::BK + et;
        if (t < te) {
          // this thread's chunk of dy and of base, at the same place in their panels
          const uint32_t ce = xp + static_cast<uint32_t>(et * TL::XROWB + bwd_slot(ec, et) * 16);
          u32x4 wd = lds_read16(ce);
          u32x4 wb = lds_read16(ce + TL::B_OFF);
          lds_wait();
          tie(wd);
          tie(wb);
          float dyv[8], bv[8], o[8];
          chunk_to_f32<DT>(__builtin_bit_cast(Chunk, wd), dyv);
          chunk_to_f32<DT>(__builtin_bit_cast(Chunk, wb), bv);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            o[e] = gb[e] * dyv[e];
            colsum[e] = __builtin_fmaf(dyv[e], bv[e], colsum[e]);
          }
          if (dbase) *reinterpret_cast<u32x4*>(dbase + t * out + ecol) = __builtin_bit_cast(u32x4, f32_to_chunk<DT>(o));
        }
      }
      slot = slot == TL::NS - 1 ? 0 : slot + 1;
    }

    // Epilogue.  The ring is free once every wave is past its last read.
    __syncthreads();
    // (1) s * sum_k B_jk E_jk over this rank block, per output column: lane l holds
    // output column 32*(wm*TMW + i) + l%32 and rank columns 32*(wn*TN + j) + 16*(l/32) + q
    const T16* Bp = static_cast<const T16*>(a.B);
    const int frow = lane & 31, fh = lane >> 5;
    float* ep = a.e_part + static_cast<int64_t>(sp) * out * r;
#pragma unroll
    for (int i = 0; i < TL::TMW; ++i) {
      const int jl = 32 * (wm * TL::TMW + i) + frow;
      const int64_t j = j0 + jl;
      float bsum = 0.0f;
#pragma unroll
      for (int jj = 0; jj < TL::TN; ++jj) {
        const int64_t k = k0 + 32 * (wn * TL::TN + jj) + 16 * fh;
        if (j < out && k < r) {
          // k + 16 <= r: r % 8 == 0 and k % 16 == 0 give whole 8-column chunks;
          // the second chunk is checked on its own
          const bool hi = k + 8 < r;
          if constexpr (TL::BASE) {
            const Chunk b0 = *reinterpret_cast<const Chunk*>(Bp + j * r + k);
            const Chunk b1 = hi ? *reinterpret_cast<const Chunk*>(Bp + j * r + k + 8) : zero_chunk();
            float bf[16];
            chunk_to_f32<DT>(b0, *reinterpret_cast<float(*)[8]>(bf));
            chunk_to_f32<DT>(b1, *reinterpret_cast<float(*)[8]>(bf + 8));
            float u0 = 0.0f, u1 = 0.0f;
#pragma unroll
            for (int q = 0; q < 16; q += 2) {
              u0 = __builtin_fmaf(bf[q], acc[i][jj][q], u0);
              u1 = __builtin_fmaf(bf[q + 1], acc[i][jj][q + 1], u1);
            }
            bsum += u0 + u1;
          }
          // this slice of E for d_B
          float* dst = ep + j * r + k;
          *reinterpret_cast<f32x4*>(dst) = f32x4{acc[i][jj][0], acc[i][jj][1], acc[i][jj][2], acc[i][jj][3]};
          *reinterpret_cast<f32x4*>(dst + 4) = f32x4{acc[i][jj][4], acc[i][jj][5], acc[i][jj][6], acc[i][jj][7]};
          if (hi) {
            *reinterpret_cast<f32x4*>(dst + 8) = f32x4{acc[i][jj][8], acc[i][jj][9], acc[i][jj][10], acc[i][jj][11]};
            *reinterpret_cast<f32x4*>(dst + 12) =
                f32x4{acc[i][jj][12], acc[i][jj][13], acc[i][jj][14], acc[i][jj][15]};
          }
        }
      }
      bsum += __shfl_xor(bsum, 32, 64);
      if (fh == 0) red[32 * 128 + wn * 128 + jl] = bsum;
    }
    if constexpr (TL::BASE) {
#pragma unroll
      for (int e = 0; e < 8; ++e) red[et * 128 + 8 * ec + e] = colsum[e];
    }
  }
  if constexpr (!TL::BASE) return;  // the plain contraction has no column sums
  // (2) the column sums of dy * base over the slice and the rank-block sums
  __syncthreads();
  if (tid < TL::BM && j0 + tid < out) {
    float bs = 0.0f, cs = 0.0f;
#pragma unroll
    for (int w = 0; w < TL::WN; ++w) bs += red[32 * 128 + w * 128 + tid];
    if (want_base)
      for (int t = 0; t < 32; ++t) cs += red[t * 128 + tid];
    a.col_part[(static_cast<int64_t>(sp) * nTl + nt) * out + j0 + tid] = cs + a.s * bs;
  }
}

// Rank block width 128*TN (TN 1..3, least padding of r, then widest) and K splits.
int bwd_tn(int64_t r) {
  int best = 1;
  int64_t best_pad = -1;
  for (int tn = 1; tn <= 3; ++tn) {
    const int64_t w = 128 * tn;
    const int64_t pad = bcdiv(std::max<int64_t>(r, 1), w) * w;
    if (best_pad < 0 || pad <= best_pad) {
      best = tn;
      best_pad = pad;
    }
  }
  return best;
}

struct BwdPlan {
  int tn = 1, nCB = 0, nTiles = 0, nSplit = 1;
  size_t off_col = 0, bytes = 0;
};

BwdPlan bwd_plan(int64_t T, int64_t out, int64_t r, bool vec) {
  BwdPlan p;
  if (!vec) return p;
  p.tn = bwd_tn(r);
  p.nCB = static_cast<int>(bcdiv(out, 128));
  p.nTiles = static_cast<int>(bcdiv(std::max<int64_t>(r, 1), 128 * p.tn));
  const int64_t blocks = static_cast<int64_t>(p.nCB) * p.nTiles;
  // about one workgroup per CU of the 256 (a workgroup holds a whole CU's
  // LDS), at least 8 stages of 32 tokens each.  Measured at T = out = 8192:
  // r = 384 (64 blocks) takes 158 us with 4 slices against 208 us with 8 and
  // 243 us with 2; 2r = 768 over 8192 rows (128 blocks) is fastest with 2.
  int64_t split = bcdiv(256, std::max<int64_t>(blocks, 1));
  split = std::min<int64_t>(split, std::max<int64_t>(1, T / 256));
  split = std::max<int64_t>(1, std::min<int64_t>(split, 64));
  p.nSplit = static_cast<int>(split);
  const size_t e_bytes = static_cast<size_t>(p.nSplit) * out * r * 4;
  p.off_col = (e_bytes + 255) & ~static_cast<size_t>(255);
  p.bytes = p.off_col + static_cast<size_t>(p.nSplit) * p.nTiles * out * 4;
  return p;
}

// Ring depth: as many stages as fit in the 160 KB of LDS, at most five (the
// 40 KB stages of the rank-384 tile with the base panel: four; the 56 KB
// stages of the rank-384 tile with dual Y panels: two).
template <int TN, bool BASE, bool DUAL, int KIND = kBwd16>
constexpr int bwd_ring() {
  constexpr int panel = 32 * 256;
  constexpr int x = KIND == kBwdX8 ? panel / 2 + 1024 : panel, base = KIND == kBwdBase8 ? panel / 2 : panel;
  constexpr int stage = x + panel * (DUAL ? 2 : 1) * TN + (BASE ? base : 0);
  constexpr int lds = 160 * 1024 - (KIND == kBwdX8 ? 2 * panel : 0);
  return lds / stage < 5 ? lds / stage : 5;
}

template <int DT, int TN, bool BASE = true, bool DUAL = false, int KIND = kBwd16>
void launch_bwd_dma(const BwdArgs& a, hipStream_t stream) {
  using TL = BwdTile<TN, bwd_ring<TN, BASE, DUAL, KIND>(), BASE, DUAL, KIND>;
  const int64_t total = static_cast<int64_t>(a.nCB) * a.nTiles * a.nSplit;
  hipLaunchKernelGGL((lora_bwd_dma<DT, TL>), dim3(static_cast<unsigned>(bcdiv(total, 8) * 8)), dim3(TL::NT), 0,
                     stream, a);
}

}  // namespace
}  // namespace dora
