// Products of 16-bit activations (or gradients) with the frozen weight in 4-bit
// blocks, for gfx950:
//
//   forward    y_tj  = sum_k x_tk W_jk,   contraction over in;
//   backward   dx_tk = sum_j g_tj W_jk,   contraction over out.
//
// A weight value leaves its 4 bits as an exact bf16 or fp16 value (the scale is a
// power of two, applied by the conversion), so the products are those of the
// 16-bit matrix instruction: exact in fp32, added in fp32, rounded once.
#include <algorithm>
#include <type_traits>

#include "dma_common.hpp"
#include "q4_common.hpp"

namespace dora {

namespace {

struct GemmArgs {
  const void* x;     // [T x K], rows of xp elements (a multiple of 8), zeros behind K
  int64_t xp;
  const uint8_t *wq, *we;
  int64_t T, N, K;
  int rt, ct;  // row and column tiles of the weight
  void* y;
  int vec;  // 16-byte stores of y
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

// Few rows, forward.  A workgroup owns one row of tiles (32 output columns) and
// 16 * NT tokens; its waves take the steps of 128 columns in turn and their sums
// meet in LDS.  The weight goes from global memory straight into the fragments of
// mfma 16x16x32: lane l holds row l % 16 of a half tile and block l / 16 of the
// four, 16 bytes, and the rows' values at the same 32 columns.
template <int DT, int NT, int NW>
__global__ __launch_bounds__(64 * NW) void q4_few(GemmArgs a) {
  using V8 = typename Dt<DT>::V8;
  using T16 = typename Dt<DT>::T;
  __shared__ f32x4 red[NW][2][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t n = lane & 15, gb = lane >> 4;
  const uint32_t rb = blockIdx.x % static_cast<uint32_t>(a.rt);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x / static_cast<uint32_t>(a.rt)) * (16 * NT);
  const uint32_t at = q4_unit(n & 3, n >> 2, gb & 1), eat = 32 * (gb & 1) + 2 * n;
  const uint8_t* wq = a.wq + static_cast<int64_t>(rb) * a.ct * kQ4TileQ + at;
  const uint8_t* we = a.we + static_cast<int64_t>(rb) * a.ct * kQ4TileE + eat;
  f32x4 acc[NT][2];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = f32x4{};
  const int steps = (a.ct + 1) / 2;
  for (int s = wave; s < steps; s += NW) {
    // past the last tile: that one again, against zeros
    const int64_t tile = min(2 * s + static_cast<int>(gb >> 1), a.ct - 1);
    const u32x4 w0 = *reinterpret_cast<const u32x4*>(wq + tile * kQ4TileQ);
    const u32x4 w1 = *reinterpret_cast<const u32x4*>(wq + tile * kQ4TileQ + 512);
    const uint32_t e = *reinterpret_cast<const uint16_t*>(we + tile * kQ4TileE);
    const float s0 = q4_scale(e & 255), s1 = q4_scale(e >> 8);
    const int64_t k = static_cast<int64_t>(s) * 128 + 32 * gb;
    Chunk x[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int64_t row = t0 + 16 * t + n;
      const T16* xr = static_cast<const T16*>(a.x) + row * a.xp + k;
#pragma unroll
      for (int m = 0; m < 4; ++m)
        x[t][m] = row < a.T && k + 8 * m < a.xp ? *reinterpret_cast<const Chunk*>(xr + 8 * m) : zero_chunk();
    }
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const V8 f0 = __builtin_bit_cast(V8, q4_decode8<DT>(w0[m], s0));
      const V8 f1 = __builtin_bit_cast(V8, q4_decode8<DT>(w1[m], s1));
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        acc[t][0] = Dt<DT>::mfma16(f0, __builtin_bit_cast(V8, x[t][m]), acc[t][0]);
        acc[t][1] = Dt<DT>::mfma16(f1, __builtin_bit_cast(V8, x[t][m]), acc[t][1]);
      }
    }
  }
  // register q of lane l is row 4 * (l / 16) + q of its half tile, for token l % 16:
  // rows 8 * (l / 16) + 0 .. 7 of the tile with the other half's
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (t > 0) __syncthreads();
    red[wave][0][lane] = acc[t][0];
    red[wave][1][lane] = acc[t][1];
    __syncthreads();
    if (wave == 0) {
      f32x4 s0 = red[0][0][lane], s1 = red[0][1][lane];
#pragma unroll
      for (int w = 1; w < NW; ++w) s0 += red[w][0][lane], s1 += red[w][1][lane];
      const float f[8] = {s0[0], s0[1], s0[2], s0[3], s1[0], s1[1], s1[2], s1[3]};
      store8<DT>(a, t0 + 16 * t + n, static_cast<int64_t>(rb) * 32 + 8 * gb, f);
    }
  }
}

// Two 16-bit values of two words: their low halves, their high halves.
__device__ inline uint32_t lows(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100u); }
__device__ inline uint32_t highs(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302u); }

// Exponents of rows 8g + i in the order of memory (i = 0, 4, 1, 5, 2, 6, 3, 7).
__device__ inline float scale_of_row(const u32x2& e, int i) {
  const uint32_t w = (i & 2) ? e[1] : e[0];
  return q4_scale((w >> (16 * (i & 1) + 8 * (i >> 2))) & 255u);
}

// Few rows, backward.  A workgroup owns 128 output columns (two tiles) and 16 * NT
// tokens; its waves take the rows of tiles in turn.  Lane l holds eight columns,
// 8 * (l % 16) .. + 7, of rows 8 * (l / 16) .. + 7: a row's eight values are
// converted with its scale, two rows' then paired by column, and fragment f has
// columns 8 n + f.
template <int DT, int NT, int NW>
__global__ __launch_bounds__(64 * NW) void q4_few_bwd(GemmArgs a) {
  using V8 = typename Dt<DT>::V8;
  using T16 = typename Dt<DT>::T;
  __shared__ f32x4 red[NW][8][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t n = lane & 15, g = lane >> 4;
  const uint32_t pairs = static_cast<uint32_t>(a.ct + 1) / 2;
  const uint32_t cb = blockIdx.x % pairs;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x / pairs) * (16 * NT);
  const uint32_t b = (n >> 2) & 1;
  const int64_t col_tile = min(static_cast<int64_t>(2 * cb + (n >> 3)), static_cast<int64_t>(a.ct - 1));
  f32x4 acc[NT][8];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int f = 0; f < 8; ++f) acc[t][f] = f32x4{};
  for (int rt = wave; rt < a.rt; rt += NW) {
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
      const int64_t row = t0 + 16 * t + n;
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
  // register q of lane l and fragment f is column 8 * (4 * (l / 16) + q) + f of token l % 16
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (t > 0) __syncthreads();
#pragma unroll
    for (int f = 0; f < 8; ++f) red[wave][f][lane] = acc[t][f];
    __syncthreads();
    // a quarter of the columns a wave
    if (wave < 4) {
      float v[8];
#pragma unroll
      for (int f = 0; f < 8; ++f) {
        v[f] = reinterpret_cast<const float*>(&red[0][f][lane])[wave];
#pragma unroll
        for (int w = 1; w < NW; ++w) v[f] += reinterpret_cast<const float*>(&red[w][f][lane])[wave];
      }
      store8<DT>(a, t0 + 16 * t + n, static_cast<int64_t>(cb) * 128 + 32 * g + 8 * wave, v);
    }
  }
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

struct GemmPlan {
  int64_t N = 0, K = 0, xp = 0;
  int64_t grid = 0;
  size_t pad = 0, bytes = 0;
};

GemmPlan gemm_plan(int64_t T, int64_t out, int64_t in, bool trans) {
  GemmPlan p;
  p.N = trans ? in : out;
  p.K = trans ? out : in;
  p.xp = q4_ceil(p.K, 8) * 8;
  p.pad = p.xp != p.K ? static_cast<size_t>(T) * p.xp * 2 : 0;
  p.bytes = p.pad;
  const int64_t groups = q4_ceil(T, 16);
  p.grid = trans ? q4_ceil(in, 128) * groups : q4_ceil(out, kQ4Rows) * groups;
  return p;
}

template <int DT>
void launch_typed(const GemmArgs& g, const GemmPlan& p, bool trans, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(p.grid));
  if (trans)
    hipLaunchKernelGGL((q4_few_bwd<DT, 1, 8>), grid, dim3(512), 0, stream, g);
  else
    hipLaunchKernelGGL((q4_few<DT, 1, 16>), grid, dim3(1024), 0, stream, g);
}

}  // namespace

size_t q4_gemm_workspace_bytes(int64_t T, int64_t out, int64_t in, bool trans) {
  return gemm_plan(T, out, in, trans).bytes;
}
int64_t q4_gemm_max_grid(int64_t T, int64_t out, int64_t in, bool trans) { return gemm_plan(T, out, in, trans).grid; }

hipError_t launch_q4_gemm(const Q4GemmArgs& p) {
  const GemmPlan plan = gemm_plan(p.T, p.out, p.in, p.trans);
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
  g.K = plan.K;
  g.rt = static_cast<int>(q4_ceil(p.out, kQ4Rows));
  g.ct = static_cast<int>(q4_ceil(p.in, kQ4Cols));
  g.y = p.y;
  g.vec = plan.N % 8 == 0 && (reinterpret_cast<uintptr_t>(p.y) & 15u) == 0;
  if (p.dtype == 0)
    launch_typed<0>(g, plan, p.trans, p.stream);
  else
    launch_typed<1>(g, plan, p.trans, p.stream);
  return hipGetLastError();
}

}  // namespace dora
