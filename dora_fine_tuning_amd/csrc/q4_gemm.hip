// Products of 16-bit activations (or gradients) with the frozen weight in 4-bit
// blocks, for gfx950:
//
//   forward    y_tj  = sum_k x_tk W_jk,   contraction over in;
//   backward   dx_tk = sum_j g_tj W_jk,   contraction over out.
//
// A weight value leaves its 4 bits as an exact bf16 or fp16 value (the scale is a
// power of two, applied by the conversion), so the products are those of the
// 16-bit matrix instruction: exact in fp32, added in fp32, rounded once.
//
// What bounds them, with whole calls in us (weights from memory for few rows):
//   1 row, 4096^2 and 27648 x 5120 (8.9 and 75 MB of weight): 5.4 and 15.4 in the
//     kernel, 4.9 TB/s of the second's bytes; the first is a launch and one latency;
//   37 rows, 27648 columns into 5120: 27.8, a ring of stages on 240 of the CUs that
//     waits for memory, and the join of 12 ranges (5.4 of it);
//   300 rows, backward of 8192^2: 50.5 (0.80 PFLOP/s), 57 % of the cycles in matrix
//     instructions; 384 rows are multiplied, by 96, and the join of 4 ranges takes 8.5;
//   8192 rows of 8192^2: 715 to 737 forward (1.5 PFLOP/s); 10240 rows, backward of
//     27648 x 5120: 1940 to 2000 (1.45 to 1.49).  Matrix instructions are busy for 77 and
//     80 % of the cycles at 1.69 and 1.75 GHz: the card's power is the limit, so that
//     what takes fewer cycles alone gives part of them back as clock.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "dma_common.hpp"
#include "q4_common.hpp"
#include "tile_units.hpp"

namespace dora {

namespace {

struct GemmArgs : TileGrid {
  const void* x;     // [T x K], rows of xp elements (a multiple of 8), zeros behind K
  int64_t xp;
  const uint8_t *wq, *we;
  int64_t T, N;
  int rt, ct;  // row and column tiles of the weight
  void* y;
  int vec;  // 16-byte stores of y
  float* part;  // sums of ranges, null where there is none to keep
};

// Eight consecutive output columns of a row, from column c on.
template <int DT>
__device__ inline void store8(const GemmArgs& a, int64_t row, int64_t c, const float (&f)[8]) {
  using T16 = typename Dt<DT>::T;
  if (row >= a.T || c >= a.N) return;
  T16* y = static_cast<T16*>(a.y) + row * a.N + c;
  if (a.vec) {  // N % 8 == 0
    *reinterpret_cast<Chunk*>(y) = f32_to_chunk<DT>(f);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < a.N) y[j] = Dt<DT>::from_f(f[j]);
  }
}

// ------------------------------------------------------------------ few rows
//
// The weight is streamed once, from global memory straight into the fragments of mfma
// 16x16x32; the rows of x come through the caches.  A workgroup owns a group of
// outputs and one of `splits` ranges of the contraction, whose steps its waves take
// in turn; their sums meet in LDS, those of the ranges in q4_few_join.

// The outputs of an entry (a register quad of lane l) of a forward group: register q
// is row 8 * (l / 16) + 4 * half + q of the row tile, for token l % 16.
template <int DT>
__device__ inline void store4(const GemmArgs& a, int64_t row, int64_t c, f32x4 v) {
  using T16 = typename Dt<DT>::T;
  typedef T16 t4 __attribute__((ext_vector_type(4)));
  if (row >= a.T || c >= a.N) return;
  T16* y = static_cast<T16*>(a.y) + row * a.N + c;
  const t4 o = {Dt<DT>::from_f(v[0]), Dt<DT>::from_f(v[1]), Dt<DT>::from_f(v[2]), Dt<DT>::from_f(v[3])};
  if (a.vec) {  // N % 8 == 0
    *reinterpret_cast<t4*>(y) = o;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (c + q < a.N) y[q] = o[q];
  }
}

// Chunk i of lane group g (of 16 lanes) changes places with chunk g of group i.
__device__ inline void turn4(Chunk (&x)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const auto a = __builtin_amdgcn_permlane32_swap(x[0].w[j], x[2].w[j], false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(x[1].w[j], x[3].w[j], false, false);
    const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    x[0].w[j] = c[0], x[1].w[j] = c[1], x[2].w[j] = d[0], x[3].w[j] = d[1];
  }
}

// Forward: R row tiles (of 32 output columns) and NT token tiles (of 16) a group,
// steps of 128 columns, U of them in registers.  Lane l holds row l % 16 of a half row
// tile and block l / 16 of the step's four, 16 bytes, and x at the same 32 columns.
// x is loaded 64 consecutive bytes of a row an instruction, each lane group a quarter
// of a block, and then turned between the groups (with each group's own block at once,
// 64 pieces of 16 bytes an instruction: 2 to 6 % slower from 32 rows on).
template <int NT_, int R_, int NW_, int U_>
struct FewFwd {
  static constexpr int NT = NT_, R = R_, NW = NW_, U = U_;
  static constexpr int ENTRIES = R * NT * 2 * 64;  // register quads of a group
};

template <int DT, class FW>
__global__ __launch_bounds__(64 * FW::NW) void q4_few(GemmArgs a) {
  using V8 = typename Dt<DT>::V8;
  using T16 = typename Dt<DT>::T;
  constexpr int NT = FW::NT, R = FW::R, NW = FW::NW, U = FW::U;
  __shared__ f32x4 red[NW][NT * 2 * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t n = lane & 15, gb = lane >> 4;
  const uint32_t groups = static_cast<uint32_t>(a.rt + R - 1) / R;
  const uint32_t grp = blockIdx.x % groups, split = blockIdx.x / groups;
  const int steps = (a.ct + 1) / 2;
  const int s0 = static_cast<int>(static_cast<int64_t>(steps) * split / a.nSplit);
  const int s1 = static_cast<int>(static_cast<int64_t>(steps) * (split + 1) / a.nSplit);
  const uint32_t at = q4_unit(n & 3, n >> 2, gb & 1), eat = 32 * (gb & 1) + 2 * n;
  const uint8_t *wq[R], *we[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {  // past the last row tile: that one again, not stored
    const int64_t rt = min(static_cast<int64_t>(grp) * R + r, static_cast<int64_t>(a.rt - 1));
    wq[r] = a.wq + rt * a.ct * kQ4TileQ + at;
    we[r] = a.we + rt * a.ct * kQ4TileE + eat;
  }
  const T16* xr[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t)  // past the last row: that one again, not stored
    xr[t] = static_cast<const T16*>(a.x) + min(static_cast<int64_t>(16 * t + n), a.T - 1) * a.xp + 8 * gb;
  f32x4 acc[R][NT][2];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[r][t][0] = acc[r][t][1] = f32x4{};
  u32x4 w[U][R][2];
  uint32_t e[U][R];
  Chunk x[U][NT][4];
  auto load = [&](auto uu, int s) {
    constexpr int u = decltype(uu)::value;
    // past the last tile: that one again, against zeros
    const int64_t tile = min(2 * s + static_cast<int>(gb >> 1), a.ct - 1);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      w[u][r][0] = *reinterpret_cast<const u32x4*>(wq[r] + tile * kQ4TileQ);
      w[u][r][1] = *reinterpret_cast<const u32x4*>(wq[r] + tile * kQ4TileQ + 512);
      e[u][r] = *reinterpret_cast<const uint16_t*>(we[r] + tile * kQ4TileE);
    }
    if (static_cast<int64_t>(s + 1) * 128 <= a.xp) {
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int m = 0; m < 4; ++m) x[u][t][m] = *reinterpret_cast<const Chunk*>(xr[t] + s * 128 + 32 * m);
    } else {  // the step that the rows end in
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int m = 0; m < 4; ++m)
          x[u][t][m] = s * 128 + 32 * m + static_cast<int>(8 * gb) < a.xp
                           ? *reinterpret_cast<const Chunk*>(xr[t] + s * 128 + 32 * m)
                           : zero_chunk();
    }
  };
  auto multiply = [&](auto uu) {
    constexpr int u = decltype(uu)::value;
#pragma unroll
    for (int t = 0; t < NT; ++t) turn4(x[u][t]);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float sc0 = q4_scale(e[u][r] & 255u), sc1 = q4_scale(e[u][r] >> 8);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const V8 f0 = __builtin_bit_cast(V8, q4_decode8<DT>(w[u][r][0][m], sc0));
        const V8 f1 = __builtin_bit_cast(V8, q4_decode8<DT>(w[u][r][1][m], sc1));
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          acc[r][t][0] = Dt<DT>::mfma16(f0, __builtin_bit_cast(V8, x[u][t][m]), acc[r][t][0]);
          acc[r][t][1] = Dt<DT>::mfma16(f1, __builtin_bit_cast(V8, x[u][t][m]), acc[r][t][1]);
        }
      }
    }
  };
  // U - 1 steps are in flight while one is multiplied
  unrolled<U - 1>([&](auto uu) {
    if (s0 + wave + decltype(uu)::value * NW < s1) load(uu, s0 + wave + decltype(uu)::value * NW);
  });
  for (int s = s0 + wave; s < s1; s += NW * U) {
    unrolled<U>([&](auto uu) {
      constexpr int u = decltype(uu)::value, nu = (u + U - 1) % U;
      if (s + u * NW < s1) {
        if (s + (u + U - 1) * NW < s1) load(std::integral_constant<int, nu>{}, s + (u + U - 1) * NW);
        __builtin_amdgcn_sched_barrier(0);
        multiply(uu);
        __builtin_amdgcn_sched_barrier(0);
      }
    });
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (r > 0) __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) red[wave][(t * 2 + h) * 64 + lane] = acc[r][t][h];
    __syncthreads();
    for (int i = threadIdx.x; i < NT * 2 * 64; i += 64 * NW) {
      f32x4 v = red[0][i];
#pragma unroll
      for (int w = 1; w < NW; ++w) v += red[w][i];
      if (a.part) {
        reinterpret_cast<f32x4*>(a.part)[(static_cast<int64_t>(blockIdx.x) * R + r) * (NT * 2 * 64) + i] = v;
      } else {
        const int l = i & 63, h = (i >> 6) & 1, t = i >> 7;
        store4<DT>(a, 16 * t + (l & 15), (static_cast<int64_t>(grp) * R + r) * 32 + 8 * (l >> 4) + 4 * h, v);
      }
    }
  }
}

// One thread an entry: its ranges' sums added in order.
template <int DT, class FW>
__global__ __launch_bounds__(256) void q4_few_join(GemmArgs a) {
  const int64_t groups = (a.rt + FW::R - 1) / FW::R, all = groups * FW::ENTRIES;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= all) return;
  const f32x4* p = reinterpret_cast<const f32x4*>(a.part) + i;
  f32x4 v = p[0];
  for (int k = 1; k < a.nSplit; ++k) v += p[k * all];
  const int64_t rt = i / (FW::NT * 2 * 64);
  const int j = static_cast<int>(i % (FW::NT * 2 * 64)), l = j & 63, h = (j >> 6) & 1, t = j >> 7;
  store4<DT>(a, 16 * t + (l & 15), rt * 32 + 8 * (l >> 4) + 4 * h, v);
}

// Two 16-bit values of two words: their low halves, their high halves.
__device__ inline uint32_t lows(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ inline uint32_t highs(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

// Exponents of rows 8g + i in the order of memory (i = 0, 4, 1, 5, 2, 6, 3, 7).
__device__ inline float scale_of_row(const u32x2& e, int i) {
  const uint32_t w = (i & 2) ? e[1] : e[0];
  return q4_scale((w >> (16 * (i & 1) + 8 * (i >> 2))) & 255u);
}

// Few rows, backward.  A group is 128 output columns (two tiles) and NT token tiles;
// a step is a row of tiles.  Lane l holds eight columns, 8 * (l % 16) .. + 7, of rows
// 8 * (l / 16) .. + 7: a row's eight values are converted with its scale, two rows' then
// paired by column, and fragment f has columns 8 n + f.
template <int NT_, int NW_>
struct FewBwd {
  static constexpr int NT = NT_, NW = NW_;
  static constexpr int ENTRIES = NT * 8 * 64;  // register quads of a group
};

// Register q of lane l of the eight fragments: columns 8 * (4 * (l / 16) + q) + 0 .. 7
// of token l % 16.
template <int DT>
__device__ inline void store_few_bwd(const GemmArgs& a, int64_t grp, int t, int q, int l, const float (&v)[8]) {
  store8<DT>(a, 16 * t + (l & 15), grp * 128 + 32 * (l >> 4) + 8 * q, v);
}

template <int DT, class FW>
__global__ __launch_bounds__(64 * FW::NW) void q4_few_bwd(GemmArgs a) {
  using V8 = typename Dt<DT>::V8;
  using T16 = typename Dt<DT>::T;
  constexpr int NT = FW::NT, NW = FW::NW;
  __shared__ f32x4 red[NW][8 * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t n = lane & 15, g = lane >> 4;
  const uint32_t groups = static_cast<uint32_t>(a.ct + 1) / 2;
  const uint32_t grp = blockIdx.x % groups, split = blockIdx.x / groups;
  const int r0 = static_cast<int>(static_cast<int64_t>(a.rt) * split / a.nSplit);
  const int r1 = static_cast<int>(static_cast<int64_t>(a.rt) * (split + 1) / a.nSplit);
  const uint32_t b = (n >> 2) & 1;
  // past the last tile: that one again, not stored
  const int64_t col_tile = min(2 * static_cast<int>(grp) + static_cast<int>(n >> 3), a.ct - 1);
  f32x4 acc[NT][8];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int f = 0; f < 8; ++f) acc[t][f] = f32x4{};
  for (int rt = r0 + wave; rt < r1; rt += NW) {
    const int64_t tile = static_cast<int64_t>(rt) * a.ct + col_tile;
    const uint8_t* wq = a.wq + tile * kQ4TileQ + 4 * (n & 3);
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = *reinterpret_cast<const uint32_t*>(wq + q4_unit(i, g, b));
    const u32x2 e = *reinterpret_cast<const u32x2*>(a.we + tile * kQ4TileE + 32 * b + 8 * g);
    const int64_t k = static_cast<int64_t>(rt) * 32 + 8 * g;
    Chunk x[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int64_t row = 16 * t + n;
      x[t] = row < a.T && k < a.xp ? *reinterpret_cast<const Chunk*>(static_cast<const T16*>(a.x) + row * a.xp + k)
                                   : zero_chunk();
    }
    Chunk p[8];  // row i's eight columns
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = q4_decode8<DT>(w[i], scale_of_row(e, i));
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      Chunk lo, hi;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        lo.w[h] = lows(p[2 * h].w[c], p[2 * h + 1].w[c]);
        hi.w[h] = highs(p[2 * h].w[c], p[2 * h + 1].w[c]);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const V8 xv = __builtin_bit_cast(V8, x[t]);
        acc[t][2 * c] = Dt<DT>::mfma16(__builtin_bit_cast(V8, lo), xv, acc[t][2 * c]);
        acc[t][2 * c + 1] = Dt<DT>::mfma16(__builtin_bit_cast(V8, hi), xv, acc[t][2 * c + 1]);
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (t > 0) __syncthreads();
#pragma unroll
    for (int f = 0; f < 8; ++f) red[wave][f * 64 + lane] = acc[t][f];
    __syncthreads();
    static_assert(NW == 8, "one register quad a thread");
    const int i = threadIdx.x;
    f32x4 v = red[0][i];
#pragma unroll
    for (int w = 1; w < NW; ++w) v += red[w][i];
    if (a.nSplit > 1) {
      reinterpret_cast<f32x4*>(a.part)[(static_cast<int64_t>(blockIdx.x) * NT + t) * (8 * 64) + i] = v;
    } else {
      red[0][i] = v;
      __syncthreads();
      if (wave < 4) {  // a quarter of the columns a wave
        float o[8];
#pragma unroll
        for (int f = 0; f < 8; ++f) o[f] = reinterpret_cast<const float*>(&red[0][f * 64 + lane])[wave];
        store_few_bwd<DT>(a, grp, t, wave, lane, o);
      }
    }
  }
}

// One thread eight columns: their ranges' sums added in order.
template <int DT, class FW>
__global__ __launch_bounds__(256) void q4_few_bwd_join(GemmArgs a) {
  const int64_t groups = (a.ct + 1) / 2, all = groups * FW::ENTRIES;
  const int64_t tile = blockIdx.x;  // of a group: its token tile
  const int q = threadIdx.x >> 6, l = threadIdx.x & 63;
  const float* p = a.part + ((tile * 8) * 64 + l) * 4 + q;
  float v[8];
#pragma unroll
  for (int f = 0; f < 8; ++f) v[f] = p[f * 256];
  for (int k = 1; k < a.nSplit; ++k)
#pragma unroll
    for (int f = 0; f < 8; ++f) v[f] += p[k * all * 4 + f * 256];
  store_few_bwd<DT>(a, tile / FW::NT, static_cast<int>(tile % FW::NT), q, l, v);
}

// ------------------------------------------------------------------ tiles
//
// Tile geometry: WM x WN waves (four), each TMW x TNW matrix tiles of 16 x 16 with their
// accumulators in registers; a ring of NS slots of one stage, 64 contraction steps
// of both operands.  x goes to LDS as rows of 128 bytes, the 16-byte chunk that lane
// group g of the reads takes in step s in place (4 s + g) ^ ((p/2) % 8) of row p: a
// read's lanes go through the banks in parties of eight rows of one group and the other
// eight of the next, and so meet 16 distinct bank groups.  (In the order 2 g + s of the
// forward's columns they met two and two: 46 % of the LDS cycles, and 741 us instead of
// 722, at 8192^2 x 8192.)  The weight's
// 4-bit tiles go as they are, 64 bytes apart from their neighbours (the backward's lanes
// read two tiles at once).
template <int WM_, int WN_, int TMW_, int TNW_, int NS_, int OCC_, bool TRANS_>
struct Q4Tile {
  static constexpr int WM = WM_, WN = WN_, TMW = TMW_, TNW = TNW_, NS = NS_, OCC = OCC_;
  static constexpr bool TRANS = TRANS_;
  static constexpr int NW = 4, NT = 256;
  static constexpr int BM = 16 * TMW * WM, BN = 16 * TNW * WN, BK = 64;
  static constexpr int WT = BN / 32, WSTEP = static_cast<int>(kQ4TileQ) + 64;  // weight tiles of a stage
  static constexpr int XQ = (BM / 8 + NW - 1) / NW;  // x rows come eight an instruction
  static constexpr int X_BYTES = XQ * NW * 1024, W_BYTES = WT * WSTEP, E_BYTES = NW * 256;
  static constexpr int SLOT_BYTES = X_BYTES + W_BYTES + E_BYTES;
  static constexpr int LDS_BYTES = NS * SLOT_BYTES;
  static constexpr int WQ = WT / NW, L = XQ + WQ + 1;  // DMA instructions a wave
  static constexpr int CT = BN / 64;  // column tiles of the backward's stage (two row tiles)
  static constexpr int NM = TMW * TNW;  // matrix instructions of a step of 32
  static constexpr int NST = NM / 2;    // 16-byte stores of a wave's tile
  static constexpr int WAIT = (NS - 2) * L;   // DMA instructions younger than the slot waited for
  static constexpr int LA = (L + 1) / 2;      // a slot's loads stand in the step after it is free and in the next one
  static constexpr int RELAX = NS - 2;        // stages whose slot was loaded before a tile's stores
  // While a wave multiplies it goes before the other workgroups' waves on its SIMD, so
  // that these convert and wait meanwhile instead of all doing the same at once: the
  // widest tile backward 7 to 12 % faster (8192^2 x 8192: 805 and 728 us), the small ones
  // 1 % on the mean; not forward in the widest, where it is 0.5 % slower.
  static constexpr bool FIRST = TRANS || TMW < 8;
  static_assert(WM * WN == NW && WQ * NW == WT, "whole DMA instructions per wave");
  static_assert(WT * 16 <= NW * 64, "exponents of a stage in one DMA instruction a wave");
  static_assert(!TRANS || TNW == 4, "a backward lane's columns");
  static_assert(TNW % 2 == 0 && NS >= 3, "pairs of half tiles; the ring");
  static_assert(WAIT + NST < 64, "vmcnt range");
  static_assert(LDS_BYTES * OCC <= 160 * 1024, "LDS");
};

template <int OFF>
__device__ inline u32x2 lds_read8_at(uint32_t base) {
  static_assert(OFF >= 0 && OFF < 65536, "ds offset field");
  u32x2 v;
  asm volatile("ds_read_b64 %0, %1 offset:%2" : "=v"(v) : "v"(base), "n"(OFF) : "memory");
  return v;
}
template <int OFF>
__device__ inline uint32_t lds_read2_at(uint32_t base) {
  static_assert(OFF >= 0 && OFF < 65536, "ds offset field");
  uint32_t v;
  asm volatile("ds_read_u16 %0, %1 offset:%2" : "=v"(v) : "v"(base), "n"(OFF) : "memory");
  return v;
}
__device__ inline void tie1(uint32_t& v) { asm volatile("" : "+v"(v)); }

// Eight output columns of a row; stores past the matrix are dropped by the buffer
// resource, so that a tile is always the same number of stores.
template <int DT>
__device__ inline void store8_to(__amdgpu_buffer_rsrc_t ry, int vec, uint32_t row, uint32_t n, uint32_t c,
                                 const float (&f)[8]) {
  const Chunk o = f32_to_chunk<DT>(f);
  const uint32_t at = (row * n + c) * 2;
  if (vec) {
    __builtin_amdgcn_raw_buffer_store_b128(u32x4{o.w[0], o.w[1], o.w[2], o.w[3]}, ry, c < n ? at : kOob, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(o.w[i >> 1] >> (16 * (i & 1))), ry,
                                            c + i < n ? at + 2 * i : kOob, 0, 0);
  }
}
// Rows [m, m + most) of y, as far as they exist.
__device__ inline __amdgpu_buffer_rsrc_t rows_of_y(const GemmArgs& a, int64_t m, int most) {
  const int64_t rows = min(max(a.T - m, int64_t(0)), static_cast<int64_t>(most));
  return buffer_of(static_cast<char*>(a.y) + (rows > 0 ? m * a.N * 2 : 0), rows * a.N * 2);
}

// The fragments of a group of matrix tiles (two forward, TNW backward) of one row of
// them, as the 16-byte pieces of y they are.  Forward: register q of half tile h is
// column 8 g + 4 h + q (g = lane / 16).  Backward: register q of fragment f is
// column 4 * (4 g + q) + f.
template <int DT, class TL>
__device__ inline void store_group(__amdgpu_buffer_rsrc_t ry, int vec, uint32_t row, int64_t N, int64_t c0, int lane,
                                   const f32x4* acc) {
  const uint32_t g = static_cast<uint32_t>(lane) >> 4, n = static_cast<uint32_t>(N), c = static_cast<uint32_t>(c0);
  if constexpr (!TL::TRANS) {
    const float f[8] = {acc[0][0], acc[0][1], acc[0][2], acc[0][3], acc[1][0], acc[1][1], acc[1][2], acc[1][3]};
    store8_to<DT>(ry, vec, row, n, c + 8 * g, f);
  } else {
#pragma unroll
    for (int q = 0; q < 4; q += 2) {
      const float f[8] = {acc[0][q],     acc[1][q],     acc[2][q],     acc[3][q],
                          acc[0][q + 1], acc[1][q + 1], acc[2][q + 1], acc[3][q + 1]};
      store8_to<DT>(ry, vec, row, n, c + 16 * g + 4 * q, f);
    }
  }
}

// Two or three workgroups a CU, each taking its units in turn (tile_units.hpp).  The ring runs
// on from one unit to the next: while a unit's last slots are worked on, the next
// one's first ones load, and its stores are under way while the next one's products
// run.  A step of 32 works on fragments that were read and converted during the step
// before: reads stand behind its first matrix instructions, the conversions behind
// its last ones.
template <int DT, class TL>
__global__ __launch_bounds__(TL::NT, TL::OCC) void q4_gemm_tile(GemmArgs a) {
  using V8 = typename Dt<DT>::V8;
  __shared__ __attribute__((aligned(1024))) char smem[TL::LDS_BYTES];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / TL::WN, wn = wave % TL::WN;
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_char_t*)smem));

  Unit cu;
  if (!unit_of(0, a, cu)) return;

  // ---- the issuing side: its unit, and that unit's buffer resources (what lies
  // past an operand reads zero; past the last unit everything does, so that every
  // step issues the same instructions and the waits count them exactly)
  const int xr = wave * 8 + (lane >> 3);  // x row of DMA instruction 0
  const int xp = (lane & 7) ^ ((xr >> 1) & 7);  // its logical chunk, in the order 4 s + g that the reads ask for
  const int xc = TL::TRANS ? xp : ((xp & 3) << 1) | (xp >> 2);
  const uint32_t xo = static_cast<uint32_t>(xr * a.xp) * 2 + 16 * xc;
  const uint32_t xstep = static_cast<uint32_t>(TL::NW * 8 * a.xp) * 2;
  const int et = (wave * 64 + lane) >> 4;  // weight tile whose exponents this lane loads
  const uint32_t rowq = static_cast<uint32_t>(a.ct) * kQ4TileQ, rowe = static_cast<uint32_t>(a.ct) * kQ4TileE;

  int ik = 0, ist = 0, iend = 0;
  bool live = true;
  __amdgpu_buffer_rsrc_t rx, rw, re;
  int in0 = 0;  // backward: the first column tile
  uint32_t xat = 0, wat[TL::WQ], eat = 0;
  auto issue_stage = [&]() {
    // columns past the row are no part of it
    xat = static_cast<int64_t>(ist) * 64 + 8 * xc < a.xp ? static_cast<uint32_t>(ist) * 128 : 0x80000000u;
    if constexpr (TL::TRANS) {
      const int64_t r0 = 2 * static_cast<int64_t>(ist), n = live ? min(max(a.rt - r0, int64_t(0)), int64_t(2)) : 0;
      rw = buffer_of(a.wq + (n > 0 ? r0 * rowq : 0), n * rowq);
      re = buffer_of(a.we + (n > 0 ? r0 * rowe : 0), n * rowe);
    } else {
#pragma unroll
      for (int q = 0; q < TL::WQ; ++q)
        wat[q] = static_cast<uint32_t>(q * TL::NW + wave) * rowq + static_cast<uint32_t>(ist) * kQ4TileQ + 16 * lane;
      eat = et < TL::WT ? static_cast<uint32_t>(et) * rowe + static_cast<uint32_t>(ist) * kQ4TileE + 4 * (lane & 15)
                        : kOob;
    }
  };
  auto issue_unit = [&](Unit u) {
    ist = u.st0;
    iend = u.st1;
    const int64_t m0 = static_cast<int64_t>(u.rb) * TL::BM;
    const int64_t xrows = live ? min(a.T - m0, static_cast<int64_t>(TL::BM)) : 0;
    rx = buffer_of(static_cast<const char*>(a.x) + m0 * a.xp * 2, xrows * a.xp * 2);
    if constexpr (TL::TRANS) {
      in0 = u.nt * TL::CT;
#pragma unroll
      for (int q = 0; q < TL::WQ; ++q) {
        const int t = q * TL::NW + wave, c = in0 + t % TL::CT;
        wat[q] = c < a.ct ? (t / TL::CT) * rowq + static_cast<uint32_t>(c) * kQ4TileQ + 16 * lane : kOob;
      }
      const int c = in0 + et % TL::CT;
      eat = et < TL::WT && c < a.ct ? (et / TL::CT) * rowe + static_cast<uint32_t>(c) * kQ4TileE + 4 * (lane & 15)
                                    : kOob;
    } else {
      const int64_t r0 = static_cast<int64_t>(u.nt) * TL::WT;
      const int64_t n = live ? min(a.rt - r0, static_cast<int64_t>(TL::WT)) : 0;
      rw = buffer_of(a.wq + r0 * rowq, n * rowq);
      re = buffer_of(a.we + r0 * rowe, n * rowe);
    }
  };
  // DMA instruction k of the issuing side's stage (k compile time)
  auto issue1 = [&](int slot, auto kk) {
    constexpr int k = decltype(kk)::value;
    char* so = smem + slot * TL::SLOT_BYTES;
    if constexpr (k < TL::XQ) {
      dma16(rx, so + (k * TL::NW + wave) * 1024, xo + k * xstep + xat);
    } else if constexpr (k < TL::XQ + TL::WQ) {
      constexpr int q = k - TL::XQ;
      dma16(rw, so + TL::X_BYTES + (q * TL::NW + wave) * TL::WSTEP, wat[q]);
    } else {
      char* d = so + TL::X_BYTES + TL::W_BYTES + wave * 256;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(re, (lds_void_t*)d, 4, eat, 0, 0, 0);
    }
  };
  auto issue_next = [&]() {  // to the next stage, or the next unit's first
    if (++ist == iend) {
      Unit u;
      live = unit_of(++ik, a, u);
      if (!live) u = Unit{0, 0, 0, 1 << 30, 0, -1};
      issue_unit(u);
    }
    issue_stage();
  };

  // ---- fragment read addresses within a slot.  Lane l holds row l % 16 of a
  // matrix tile and eight contraction steps.  Forward, step s: columns 16 g + 8 s
  // (g = l / 16), half a block's 16 bytes of the weight for both steps of the stage.
  // Backward, step s: rows 8 g of the stage's row tile s.
  const int l16 = lane & 15, g = lane >> 4;
  uint32_t xa[2];
#pragma unroll
  for (int s = 0; s < 2; ++s)
    xa[s] = lds0 + static_cast<uint32_t>((wm * TL::TMW * 16 + l16) * 128 + 16 * ((4 * s + g) ^ ((l16 >> 1) & 7)));
  const uint32_t w0 = lds0 + TL::X_BYTES, e0 = w0 + TL::W_BYTES;
  uint32_t wa[TL::TRANS ? 2 : 1], ea;
  if constexpr (TL::TRANS) {
    const int col = wn * TL::TNW * 16 + TL::TNW * l16;  // the lane's first column of the tile
    const int t = col >> 6, b = (col >> 5) & 1;
#pragma unroll
    for (int h = 0; h < 2; ++h)  // rows 8g + i with (i / 2) % 2 == h
      wa[h] = w0 + static_cast<uint32_t>(t * TL::WSTEP) + q4_unit(2 * h, g, b) - 256 * h + ((col >> 1) & 15);
    ea = e0 + static_cast<uint32_t>(t * 64 + 32 * b + 8 * g);
  } else {
    wa[0] = w0 + static_cast<uint32_t>(wn * TL::TNW / 2 * TL::WSTEP) + q4_unit(l16 & 3, l16 >> 2, g >> 1) + 8 * (g & 1);
    ea = e0 + static_cast<uint32_t>(wn * TL::TNW / 2 * 64 + 32 * (g >> 1) + 2 * l16);
  }

  f32x4 acc[TL::TMW][TL::TNW];
  u32x4 fx[2][TL::TMW], fw[2][TL::TNW];  // fragments of the two steps of a stage
  u32x2 rawf[TL::TRANS ? 1 : TL::TNW];   // forward: the stage's weight, both steps
  uint32_t rawe[TL::TRANS ? 1 : TL::TNW / 2];
  uint32_t rawb[TL::TRANS ? 8 : 1];      // backward: the next step's
  u32x2 rawbe;
  float scale[8];
  constexpr int NRX = TL::TMW, NRW = TL::TRANS ? 9 : TL::TNW + TL::TNW / 2;
  // Read n of the step before step s: first the weight (forward: once a stage).
  auto read1 = [&](uint32_t so, auto ss, auto nn) {
    constexpr int s = decltype(ss)::value;
    constexpr int n = decltype(nn)::value - ((TL::TRANS || s == 0) ? NRW : 0);
    if constexpr (n >= 0) {
      fx[s][n] = lds_read16_at<n * 16 * 128>(xa[s] + so);
    } else if constexpr (TL::TRANS) {
      constexpr int i = n + NRW;
      constexpr int st = s * TL::CT * TL::WSTEP;
      if constexpr (i == 8)
        rawbe = lds_read8_at<s * TL::CT * 64>(ea + so);
      else
        rawb[i] = lds_read2_at<st + 128 * i>(wa[(i >> 1) & 1] + so);
    } else {
      constexpr int j = n + NRW;
      if constexpr (j < TL::TNW)
        rawf[j] = lds_read8_at<(j / 2) * TL::WSTEP + (j % 2) * 512>(wa[0] + so);
      else
        rawe[j - TL::TNW] = lds_read2_at<(j - TL::TNW) * 64>(ea + so);
    }
  };
  // after lds_wait()
  auto tie_reads = [&](auto ss) {
    constexpr int s = decltype(ss)::value;
#pragma unroll
    for (int i = 0; i < TL::TMW; ++i) tie(fx[s][i]);
    if constexpr (TL::TRANS) {
#pragma unroll
      for (int i = 0; i < 8; ++i) tie1(rawb[i]);
      tie2(rawbe);
    } else if constexpr (s == 0) {
#pragma unroll
      for (int j = 0; j < TL::TNW; ++j) tie2(rawf[j]);
#pragma unroll
      for (int j = 0; j < TL::TNW / 2; ++j) tie1(rawe[j]);
    }
  };
  // Conversion piece p of step s: forward a fragment, backward the two of a pair of
  // columns.
  constexpr int NP = TL::TRANS ? TL::TNW / 2 : TL::TNW;
  auto convert1 = [&](auto ss, auto pp) {
    constexpr int s = decltype(ss)::value, p = decltype(pp)::value;
    if constexpr (TL::TRANS) {
      if constexpr (p == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) scale[i] = scale_of_row(rawbe, i);
      }
      uint32_t v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = q4_decode2<DT, p>(rawb[i], scale[i]);
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        fw[s][2 * p][h] = lows(v[2 * h], v[2 * h + 1]);
        fw[s][2 * p + 1][h] = highs(v[2 * h], v[2 * h + 1]);
      }
    } else {
      const uint32_t e = rawe[p / 2];
      const float sc = q4_scale(p % 2 ? e >> 8 : e & 255u);
      fw[s][p] = __builtin_bit_cast(u32x4, q4_decode8<DT>(rawf[p][s], sc));
    }
  };
  // The accumulators are named here, so the products above stay above (the
  // compiler would otherwise sink them past the barrier to their next use).
  auto pin_acc = [&]() {
#pragma unroll
    for (int i = 0; i < TL::TMW; ++i)
#pragma unroll
      for (int j = 0; j < TL::TNW; ++j) asm volatile("" : "+a"(acc[i][j]));
  };
  // An accumulator is cleared by a product of zeros, which takes its zero addend as
  // an inline constant.
  auto clear = [&](int i, int j) {
    uint32_t z = 0;
    asm volatile("" : "+v"(z));
    const V8 zv = __builtin_bit_cast(V8, u32x4{z, z, z, z});
    acc[i][j] = Dt<DT>::mfma16(zv, zv, f32x4{});
    asm volatile("" : "+a"(acc[i][j]));
  };

  // ---- fill the ring
  issue_unit(cu);
  issue_stage();
#pragma unroll
  for (int s = 0; s < TL::NS; ++s) {
    if (s + 1 < TL::NS) {
      unrolled<TL::L>([&](auto kk) { issue1(s, kk); });
      issue_next();
    } else {
      unrolled<TL::LA>([&](auto kk) { issue1(s, kk); });
    }
  }
  wait_vmcnt<(TL::NS - 2) * TL::L + TL::LA>();
  __builtin_amdgcn_s_barrier();
  using S0 = std::integral_constant<int, 0>;
  using S1 = std::integral_constant<int, 1>;
  unrolled<NRX + NRW>([&](auto nn) { read1(0u, S0{}, nn); });
  lds_wait();
  tie_reads(S0{});
  unrolled<NP>([&](auto pp) { convert1(S0{}, pp); });

  int ck = 0;
  bool more = false;
  auto look_ahead = [&]() {
    Unit n;
    more = unit_of(ck + 1, a, n);
  };
  look_ahead();
#pragma unroll
  for (int i = 0; i < TL::TMW; ++i)
#pragma unroll
    for (int j = 0; j < TL::TNW; ++j) clear(i, j);

  // The products of step s, while the other step's fragments (of the slot at rd) come
  // in and the issuing side's loads into slot wr go out.
  constexpr int NM = TL::NM, MID = NM / 2;
  auto step = [&](auto ss, uint32_t rd, int wr) {
    constexpr int s = decltype(ss)::value, o = 1 - s;
    using O = std::integral_constant<int, o>;
    constexpr int NR = NRX + ((TL::TRANS || o == 0) ? NRW : 0);
    constexpr int RA = (NR + MID - 1) / MID;
    if constexpr (TL::FIRST) __builtin_amdgcn_s_setprio(1);
    constexpr int k0 = s == 1 ? 0 : TL::LA, k1 = s == 1 ? TL::LA : TL::L, DA = (k1 - k0 + NM - 1) / NM;
    unrolled<NM>([&](auto mm) {
      constexpr int m = decltype(mm)::value;
      constexpr int i = m % TL::TMW, j = m / TL::TMW;
      acc[i][j] = Dt<DT>::mfma16(__builtin_bit_cast(V8, fw[s][j]), __builtin_bit_cast(V8, fx[s][i]), acc[i][j]);
      unrolled<RA>([&](auto rr) {
        constexpr int n = m * RA + decltype(rr)::value;
        if constexpr (m < MID && n < NR) read1(rd, O{}, std::integral_constant<int, n>{});
      });
      unrolled<DA>([&](auto dd) {
        constexpr int k = k0 + m * DA + decltype(dd)::value;
        if constexpr (k < k1) issue1(wr, std::integral_constant<int, k>{});
      });
      if constexpr (m == MID) {
        lds_wait();
        tie_reads(O{});
      }
      if constexpr (m >= MID) {  // piece p behind instruction MID + p (NM - MID) / NP
        unrolled<NP>([&](auto pp) {
          constexpr int p = decltype(pp)::value;
          if constexpr (MID + p * (NM - MID) / NP == m) convert1(O{}, pp);
        });
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    if constexpr (TL::FIRST) __builtin_amdgcn_s_setprio(0);
    pin_acc();
  };

  int st = cu.st0, slot = 0;
  int relax = 0;  // stages until the last tile's stores must be done
  while (true) {
    const int s1 = slot + 1 == TL::NS ? 0 : slot + 1;
    const bool last = st + 1 == cu.st1;
    step(S0{}, static_cast<uint32_t>(slot * TL::SLOT_BYTES), slot == 0 ? TL::NS - 1 : slot - 1);
    issue_next();
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
    step(S1{}, static_cast<uint32_t>(s1 * TL::SLOT_BYTES), slot);
    slot = s1;
    ++st;
    if (!last) continue;

    // lane coordinates taken anew, so that nothing but the accumulators and the
    // loop's own values is live across the loop
    int el = static_cast<int>(threadIdx.x) & 63;
    asm volatile("" : "+v"(el));
    const uint32_t er = static_cast<uint32_t>(el & 15);
    const bool part = cu.tail >= 0 && a.part != nullptr;
    // a split's fp32 tile: 16 bytes a lane, in the order the join reads it
    const int64_t tile = static_cast<int64_t>(cu.split) * (a.nRB * a.nTiles - a.whole) + cu.tail;
    f32x4* p = reinterpret_cast<f32x4*>(a.part) + (tile * TL::NW + wave) * (NM * 64) + el;
    const int64_t m0 = static_cast<int64_t>(cu.rb) * TL::BM + wm * TL::TMW * 16;
    const __amdgpu_buffer_rsrc_t ry = rows_of_y(a, m0, TL::TMW * 16);
    const int64_t c0 = static_cast<int64_t>(cu.nt) * TL::BN + wn * TL::TNW * 16;
    constexpr int GJ = TL::TRANS ? TL::TNW : 2;
#pragma unroll
    for (int i = 0; i < TL::TMW; ++i)
#pragma unroll
      for (int j = 0; j < TL::TNW; j += GJ) {
        // one group at a time leaves the accumulator registers
#pragma unroll
        for (int q = 0; q < GJ; ++q) asm volatile("" : "+a"(acc[i][j + q]));
        if (part) {
          if (m0 + i * 16 < a.T)
#pragma unroll
            for (int q = 0; q < GJ; ++q) p[(i * TL::TNW + j + q) * 64] = acc[i][j + q];
        } else {
          store_group<DT, TL>(ry, a.vec, i * 16 + er, a.N, c0 + j * 16, el, &acc[i][j]);
        }
#pragma unroll
        for (int q = 0; q < GJ; ++q) clear(i, j + q);
      }
    if (!part && a.vec)
      relax = TL::RELAX;
    else
      wait_vmcnt<0>();
    if (!more) break;
    ++ck;
    unit_of(ck, a, cu);
    look_ahead();
    st = cu.st0;
  }
  wait_vmcnt<0>();  // the DMA past the last unit is done before the workgroup's LDS is given up
}

// One wave a group of matrix tiles of the output: its splits' sums added in order.
template <int DT, class TL>
__global__ __launch_bounds__(256) void q4_gemm_join(GemmArgs a) {
  const int lane = threadIdx.x & 63;
  constexpr int GJ = TL::TRANS ? TL::TNW : 2, PT = TL::NW * TL::NM / GJ;  // groups of a workgroup tile
  const int64_t ntail = static_cast<int64_t>(a.nRB) * a.nTiles - a.whole;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (w >= ntail * PT) return;
  const int64_t tail = w / PT;
  const int sub = static_cast<int>(w % PT) * GJ;  // its first matrix tile
  const int wave = sub / TL::NM, ij = sub % TL::NM, i = ij / TL::TNW, j = ij % TL::TNW;
  int rb, nt;
  tile_of(static_cast<uint32_t>(a.whole + tail), a, rb, nt);
  const int wm = wave / TL::WN, wn = wave % TL::WN;
  const int64_t m = static_cast<int64_t>(rb) * TL::BM + (wm * TL::TMW + i) * 16;
  if (m >= a.T) return;  // rows past the last: not written either
  const f32x4* p = reinterpret_cast<const f32x4*>(a.part) + (tail * TL::NW * TL::NM + sub) * 64 + lane;
  f32x4 s[GJ];
#pragma unroll
  for (int q = 0; q < GJ; ++q) s[q] = p[q * 64];
  for (int k = 1; k < a.nSplit; ++k) {
    const f32x4* pk = p + static_cast<int64_t>(k) * ntail * TL::NW * TL::NM * 64;
#pragma unroll
    for (int q = 0; q < GJ; ++q) s[q] += pk[q * 64];
  }
  store_group<DT, TL>(rows_of_y(a, m, 16), a.vec, static_cast<uint32_t>(lane & 15), a.N,
                      static_cast<int64_t>(nt) * TL::BN + (wn * TL::TNW + j) * 16, lane, s);
}

// An empty contraction: zeros (the kernels above need at least one step).
__global__ __launch_bounds__(256) void q4_zero(uint16_t* y, int64_t n) {
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < n;
       e += static_cast<int64_t>(gridDim.x) * 256)
    y[e] = 0;
}

// Rows that are no multiple of 8 elements, copied with zeros behind them.
__global__ __launch_bounds__(256) void q4_pad_rows(const uint16_t* x, int64_t T, int64_t K, int64_t xp, uint16_t* p) {
  const int64_t chunks = T * (xp / 8);
  for (int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; c < chunks;
       c += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t row = c / (xp / 8), k = (c - row * (xp / 8)) * 8;
    const uint16_t* s = x + row * K + k;
    uint16_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = k + j < K ? s[j] : static_cast<uint16_t>(0);
    Chunk o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o.w[j] = v[2 * j] | static_cast<uint32_t>(v[2 * j + 1]) << 16;
    *reinterpret_cast<Chunk*>(p + c * 8) = o;
  }
}

// Two or three workgroups a CU, with a wave an SIMD each, whose waits the others' work
// covers.  (A workgroup of 256 x 256 a CU, in us at 8192^2 x 8192: 734 forward and 854
// backward, against 741 and 806 of 128 x 256, both before the steps above; a workgroup of
// 64 x 256 a CU, with a ring of twice the slots, took 8 to 12 % longer than two.)
template <bool TRANS>
using WideTile = Q4Tile<1, 4, 8, 4, 3, 2, TRANS>;  // 128 x 256
template <bool TRANS>
using BroadTile = Q4Tile<1, 4, 6, 4, 3, 2, TRANS>;  // 96 x 256
template <bool TRANS>
using FlatTile = Q4Tile<1, 4, 4, 4, 4, 2, TRANS>;  // 64 x 256
template <bool TRANS>
using ThinTile = Q4Tile<1, 4, 3, 4, 4, 2, TRANS>;  // 48 x 256
template <bool TRANS>
using LowTile = Q4Tile<2, 2, 2, 4, 3, 3, TRANS>;  // 64 x 128

// Few rows: groups of R row tiles (forward) or 128 columns (backward), each in so many
// ranges of the contraction.
void few_plan(Q4Plan& p, int64_t T, int64_t out, int64_t in, bool trans, int R, int splits) {
  const int64_t groups = trans ? q4_ceil(in, 128) : q4_ceil(q4_ceil(out, kQ4Rows), R);
  p.path = Q4Plan::kFew;
  p.R = R;
  p.nSplit = splits;
  p.grid = groups * splits;
  const int64_t entries = (trans ? 8 : 2 * R) * 64 * q4_ceil(T, 16);  // register quads of a group
  p.bytes = splits > 1 ? static_cast<size_t>(p.grid * entries) * 16 : 0;
}

// Expected microseconds of few rows: the weight's and the rows' bytes into the CUs, and
// the steps that a workgroup's waves take one after the other (as long as its matrix
// tiles and rows ask for, with as many workgroups on a CU as its registers allow), of
// which the longer hides most of the other; for ranges also the join's launch, its sums
// and the partial sums written and read.
double few_us(const Q4Plan& p, int64_t T, int64_t out, int64_t in, bool trans) {
  const int64_t nt = q4_ceil(T, 16), groups = p.grid / p.nSplit;
  const double w_mb = static_cast<double>(out) * in * 17e-6 / 32, x_mb = 2e-6 * groups * T * p.K;
  const double part_mb = static_cast<double>(p.bytes) * 1e-6;
  if (trans) {
    const int64_t steps = q4_ceil(q4_ceil(q4_ceil(out, kQ4Rows), p.nSplit), 8);
    return 2.65 + 0.104 * (w_mb + 0.34 * x_mb) + q4_ceil(p.grid, 2 * kCUs) * steps * (0.351 + 0.218 * nt) +
           (p.nSplit > 1 ? 1.13 + 0.43 * p.nSplit + 0.42 * part_mb : 0.0);
  }
  const int64_t rnt = p.R * nt, steps = q4_ceil(q4_ceil(q4_ceil(in, 128), p.nSplit), rnt == 1 ? 16 : 8);
  const int64_t rounds = q4_ceil(p.grid, (rnt == 2 ? 2 : 1) * kCUs);
  const double load = 0.163 * w_mb + 0.074 * x_mb;
  const double work = static_cast<double>(rounds * steps) * (0.570 + 0.229 * rnt + 0.315 * nt);
  return 2.78 + std::cbrt(load * load * load + work * work * work) +
         (p.nSplit > 1 ? 1.50 + 0.156 * p.nSplit + 0.687 * part_mb : 0.0);
}

constexpr int kTileGroup = 8;  // column tiles of a group of the tile order

struct TileKind {
  Q4Plan::Path path;
  int64_t bm, bn, occ;
  double us[2][3];  // a stage forward and backward, with one to three workgroups on a CU
};
constexpr TileKind kTiles[] = {  // in the order of Q4Plan::Path
    {Q4Plan::kLow, 64, 128, 3, {{0.372, 0.490, 0.691}, {0.591, 0.805, 0.959}}},
    {Q4Plan::kThin, 48, 256, 2, {{0.445, 0.602, 0.0}, {0.663, 0.813, 0.0}}},
    {Q4Plan::kFlat, 64, 256, 2, {{0.508, 0.721, 0.0}, {0.703, 0.905, 0.0}}},
    {Q4Plan::kBroad, 96, 256, 2, {{0.650, 1.024, 0.0}, {0.863, 1.108, 0.0}}},
    {Q4Plan::kWide, 128, 256, 2, {{0.756, 1.350, 0.0}, {0.993, 1.368, 0.0}}},
};

// Tiles of one kind: as many rounds of one whole tile a workgroup as there are, and the
// rest in up to 16 ranges of stages each (at least four stages), whichever number is
// expected to be fastest.  Returns the expected microseconds.
double tile_us(Q4Plan& p, int64_t T, const TileKind& t, bool trans) {
  const double* us = t.us[trans ? 1 : 0];
  const int64_t slots = kCUs * t.occ;
  p.path = t.path;
  p.nRB = q4_ceil(T, t.bm);
  p.nTiles = q4_ceil(p.N, t.bn);
  const int64_t tiles = p.nRB * p.nTiles, rounds = tiles / slots, rest = tiles - rounds * slots;
  p.whole = rounds * slots;
  p.nSplit = 1;
  double least = 0.0;
  // a tile's rows that exist are written, on the mean of the tiles
  const double mb = static_cast<double>(rest) * t.bn * 4e-6 * static_cast<double>(T) / static_cast<double>(p.nRB);
  for (int s = 1; rest > 0 && s <= 16 && (s == 1 || p.S / s >= 4); ++s) {
    double c = s > 1 ? 2.53 + 0.29 * s + 0.25 * mb * s : 0.0;
    for (int64_t left = rest * s; left > 0; left -= slots)
      c += static_cast<double>(q4_ceil(p.S, s)) * us[q4_ceil(std::min(left, slots), kCUs) - 1];
    if (s == 1 || c < least) least = c, p.nSplit = s;
  }
  p.grid = std::min<int64_t>(slots, q4_ceil(p.whole + rest * p.nSplit, 8) * 8);
  p.bytes = p.nSplit > 1 ? static_cast<size_t>(rest) * p.nSplit * t.bm * t.bn * 4 : 0;
  return 4.9 + static_cast<double>(rounds) * p.S * us[t.occ - 1] + least;
}

template <int DT, class TL>
void launch_tile(const GemmArgs& g, const Q4Plan& p, hipStream_t stream) {
  hipLaunchKernelGGL((q4_gemm_tile<DT, TL>), dim3(static_cast<unsigned>(p.grid)), dim3(TL::NT), 0, stream, g);
  if (p.nSplit > 1 && !p.parts) {
    const int64_t waves = (p.nRB * p.nTiles - p.whole) * TL::NW * TL::NM / (TL::TRANS ? TL::TNW : 2);
    hipLaunchKernelGGL((q4_gemm_join<DT, TL>), dim3(static_cast<unsigned>(q4_ceil(waves, 4))), dim3(256), 0, stream, g);
  }
}

template <int DT, class FW>
void launch_few_as(const GemmArgs& g, const Q4Plan& p, hipStream_t stream) {
  hipLaunchKernelGGL((q4_few<DT, FW>), dim3(static_cast<unsigned>(p.grid)), dim3(64 * FW::NW), 0, stream, g);
  if (p.nSplit > 1 && !p.parts) {
    const dim3 grid(static_cast<unsigned>(q4_ceil(p.grid / p.nSplit * FW::ENTRIES, 256)));
    hipLaunchKernelGGL((q4_few_join<DT, FW>), grid, dim3(256), 0, stream, g);
  }
}
template <int DT, int NT>
void launch_few_nt(const GemmArgs& g, const Q4Plan& p, hipStream_t stream) {
  switch (p.R) {
    case 1:
      return launch_few_as<DT, FewFwd<NT, 1, NT == 1 ? 16 : 8, 2>>(g, p, stream);
    case 2:
      return launch_few_as<DT, FewFwd<NT, 2, 8, 2>>(g, p, stream);
    default:
      if constexpr (NT <= 2) return launch_few_as<DT, FewFwd<NT, 4, 8, 2>>(g, p, stream);
  }
}
template <int DT, int NT>
void launch_few_bwd(const GemmArgs& g, const Q4Plan& p, hipStream_t stream) {
  using FW = FewBwd<NT, 8>;
  hipLaunchKernelGGL((q4_few_bwd<DT, FW>), dim3(static_cast<unsigned>(p.grid)), dim3(64 * FW::NW), 0, stream, g);
  if (p.nSplit > 1)
    hipLaunchKernelGGL((q4_few_bwd_join<DT, FW>), dim3(static_cast<unsigned>(p.grid / p.nSplit * NT)), dim3(256), 0,
                       stream, g);
}
template <int DT, bool TRANS>
void launch_few(const GemmArgs& g, const Q4Plan& p, hipStream_t stream) {
  const int nt = static_cast<int>((g.T + 15) / 16);
  if constexpr (TRANS)
    return nt == 1 ? launch_few_bwd<DT, 1>(g, p, stream) : launch_few_bwd<DT, 2>(g, p, stream);
  else
    return nt == 1   ? launch_few_nt<DT, 1>(g, p, stream)
           : nt == 2 ? launch_few_nt<DT, 2>(g, p, stream)
                     : launch_few_nt<DT, 3>(g, p, stream);
}

template <int DT, bool TRANS>
void launch_typed(const GemmArgs& g, const Q4Plan& p, hipStream_t stream) {
  switch (p.path) {
    case Q4Plan::kFew:
      return launch_few<DT, TRANS>(g, p, stream);
    case Q4Plan::kLow:
      return launch_tile<DT, LowTile<TRANS>>(g, p, stream);
    case Q4Plan::kThin:
      return launch_tile<DT, ThinTile<TRANS>>(g, p, stream);
    case Q4Plan::kFlat:
      return launch_tile<DT, FlatTile<TRANS>>(g, p, stream);
    case Q4Plan::kBroad:
      return launch_tile<DT, BroadTile<TRANS>>(g, p, stream);
    case Q4Plan::kWide:
      return launch_tile<DT, WideTile<TRANS>>(g, p, stream);
  }
}

}  // namespace

// The kernel, its tile and its ranges are those expected to be fastest.  The times are
// fitted to 15263 calls (nine weights from 512 x 512 to 27648 x 5120, both directions, 1
// to 8192 rows, every kind with up to 16 ranges, weights out of the caches); over them
// the plan's call takes 1.0 % more than the fastest measured one on the mean with the
// tiles (12 % at most) and 3.1 % forward, 1.2 % backward with the kernels for few rows
// (29 and 20 % at most, both with 32 rows).
Q4Plan q4_plan(int64_t T, int64_t out, int64_t in, bool trans) {
  Q4Plan p;
  p.N = trans ? in : out;
  p.K = trans ? out : in;
  p.xp = q4_ceil(p.K, 8) * 8;
  p.pad = p.xp != p.K ? (static_cast<size_t>(T) * p.xp * 2 + 255) / 256 * 256 : 0;
  p.S = static_cast<int>(q4_ceil(p.K, kQ4Cols));
  Q4Plan best;
  double least = -1.0;
  auto take = [&](const Q4Plan& q, double us) {
    if (least < 0.0 || us < least) least = us, best = q;
  };
  if (T <= (trans ? 32 : 48)) {
    for (int R = 1; R <= (trans ? 1 : T <= 32 ? 4 : 2); R *= 2)
      for (int splits : {1, 2, 3, 4, 6, 8, 12, 16}) {
        if (splits > 1 && p.S / splits < 8) break;
        Q4Plan q = p;
        few_plan(q, T, out, in, trans, R, splits);
        take(q, few_us(q, T, out, in, trans));
      }
  }
  for (const TileKind& t : kTiles) {
    Q4Plan q = p;
    const double us = tile_us(q, T, t, trans);
    take(q, us);
  }
  return best;
}

void q4_plan_numbers(const Q4Plan& p, bool trans, int64_t* n) {
  const bool few = p.path == Q4Plan::kFew;
  n[0] = few ? 0 : kTiles[p.path].bm;
  n[1] = !few ? kTiles[p.path].bn : trans ? 128 : p.R * kQ4Rows;
  n[2] = p.whole;
  n[3] = few ? p.grid / p.nSplit : p.nRB * p.nTiles - p.whole;
  n[4] = p.nSplit;
  n[5] = p.grid;
}

// The plan of a forward product whose sums all stay in the workspace: as many ranges as
// the product's plan has where it splits every tile, else one.
Q4Plan q4_parts_plan(Q4Plan p, int64_t T) {
  p.parts = true;
  if (p.path == Q4Plan::kFew) {
    p.bytes = static_cast<size_t>(p.grid) * 2 * p.R * 64 * q4_ceil(T, 16) * 16;
    return p;
  }
  const TileKind& t = kTiles[p.path];
  const int64_t tiles = p.nRB * p.nTiles;
  if (p.whole > 0) p.nSplit = 1;
  p.whole = 0;
  p.grid = std::min<int64_t>(kCUs * t.occ, q4_ceil(tiles * p.nSplit, 8) * 8);
  p.bytes = static_cast<size_t>(tiles) * p.nSplit * t.bm * t.bn * 4;
  return p;
}

Q4Parts q4_parts_of(const Q4Plan& p, int64_t T) {
  Q4Parts a{};
  a.nSplit = p.nSplit;
  a.few = p.path == Q4Plan::kFew;
  if (a.few) {
    a.R = p.R;
    a.NT = static_cast<int>(q4_ceil(T, 16));
    a.all = p.grid / p.nSplit;
    return a;
  }
  auto of = [&](auto tl) {
    using TL = decltype(tl);
    a.WM = TL::WM, a.WN = TL::WN, a.TMW = TL::TMW, a.TNW = TL::TNW;
  };
  switch (p.path) {
    case Q4Plan::kLow:
      of(LowTile<false>{});
      break;
    case Q4Plan::kThin:
      of(ThinTile<false>{});
      break;
    case Q4Plan::kFlat:
      of(FlatTile<false>{});
      break;
    case Q4Plan::kBroad:
      of(BroadTile<false>{});
      break;
    default:
      of(WideTile<false>{});
  }
  a.all = p.nRB * p.nTiles;
  a.nRB = static_cast<int>(p.nRB);
  a.nTiles = static_cast<int>(p.nTiles);
  a.group = kTileGroup;
  return a;
}

hipError_t launch_q4_gemm(const Q4GemmArgs& p, const Q4Plan& plan) {
  if (plan.K == 0) {
    const int64_t n = p.T * plan.N;
    hipLaunchKernelGGL(q4_zero, dim3(static_cast<unsigned>(std::min<int64_t>(q4_ceil(n, 256), 4096))), dim3(256), 0,
                       p.stream, static_cast<uint16_t*>(p.y), n);
    return hipGetLastError();
  }
  GemmArgs g{};
  g.x = p.x;
  g.xp = plan.xp;
  if (plan.pad) {
    const int64_t chunks = p.T * (plan.xp / 8);
    hipLaunchKernelGGL(q4_pad_rows, dim3(static_cast<unsigned>(std::min<int64_t>(q4_ceil(chunks, 256), 16384))),
                       dim3(256), 0, p.stream, static_cast<const uint16_t*>(p.x), p.T, plan.K, plan.xp,
                       static_cast<uint16_t*>(p.ws));
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    g.x = p.ws;
  }
  g.wq = static_cast<const uint8_t*>(p.wq);
  g.we = static_cast<const uint8_t*>(p.we);
  g.T = p.T;
  g.N = plan.N;
  g.rt = static_cast<int>(q4_ceil(p.out, kQ4Rows));
  g.ct = static_cast<int>(q4_ceil(p.in, kQ4Cols));
  g.S = plan.S;
  g.nRB = static_cast<int>(plan.nRB);
  g.nTiles = static_cast<int>(plan.nTiles);
  g.nSplit = plan.nSplit;
  g.whole = static_cast<int>(plan.whole);
  g.group = kTileGroup;
  g.y = p.y;
  g.vec = plan.N % 8 == 0 && (reinterpret_cast<uintptr_t>(p.y) & 15u) == 0;
  g.part = plan.bytes > 0 ? reinterpret_cast<float*>(static_cast<char*>(p.ws) + plan.pad) : nullptr;
  if (p.dtype == 0)
    p.trans ? launch_typed<0, true>(g, plan, p.stream) : launch_typed<0, false>(g, plan, p.stream);
  else
    p.trans ? launch_typed<1, true>(g, plan, p.stream) : launch_typed<1, false>(g, plan, p.stream);
  return hipGetLastError();
}

}  // namespace dora
