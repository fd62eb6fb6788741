// The factored norm of a 4-bit weight with a cached base term, for gfx950:
//
//   n_i = sqrt(c_i + 2 s sum_j B_ij U_ij),  U = W A^T + (s/2) B (A A^T),
//
// c_i = ||W_i||^2.  W A^T is the forward product on the r rows of A, whose fp32 sums
// stay in the workspace as its kernels leave them (q4_gemm.hip): 17/32 bytes an element
// of W are read instead of the 5 that unpacking to 16 bits, and reading that, take.
// (s/2) A A^T comes as two 16-bit matrices from the 16-bit norm's Gram kernels (norm.hip).
#include "q4_common.hpp"

namespace dora {

namespace {

struct JoinArgs : Q4NormArgs, Q4Parts {};

// The entry of row tile rt (32 outputs), 16 rows tt of A, half h, range 0.
__device__ inline int64_t entry_of(const Q4Parts& a, int64_t rt, int tt, int h) {
  if (a.few) return (rt * a.NT + tt) * 2 + h;  // rt = group * R + its row tile
  const int mt = a.WM * a.TMW, nt = a.WN * a.TNW;  // matrix tiles of a tile
  const int rb = tt / mt, wm = tt % mt / a.TMW, i = tt % a.TMW;
  const int ct = static_cast<int>(2 * rt / nt), j = static_cast<int>(2 * rt % nt), wn = j / a.TNW;
  // the tile's number in the order of tile_units.hpp
  const int grp = ct / a.group, gn = min(a.group, a.nTiles - grp * a.group);
  const int64_t v = static_cast<int64_t>(grp) * a.group * a.nRB + rb * gn + ct % a.group;
  return (v * a.WM * a.WN + wm * a.WN + wn) * (a.TMW * a.TNW) + i * a.TNW + j % a.TNW + h;
}

// A workgroup 32 outputs, a wave every fourth 16 rows of A: B's rows times (s/2) A A^T by
// the matrix instruction in the layout of the entries, these added in the order of their
// ranges, and the dot with B.
template <int DT>
__global__ __launch_bounds__(256) void q4_norm_join(JoinArgs a) {
  using T16 = typename Dt<DT>::T;
  using V8 = typename Dt<DT>::V8;
  __shared__ float red[4][32];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, g = lane >> 4;
  const int64_t rt = blockIdx.x, c0 = rt * 32;
  const int r = static_cast<int>(a.r);
  const T16* B = static_cast<const T16*>(a.B);
  const T16 *ghi = static_cast<const T16*>(a.ghi), *glo = static_cast<const T16*>(a.glo);
  const int64_t stride = a.all * (a.few ? a.R * a.NT * 2 : a.WM * a.WN * a.TMW * a.TNW) * 64;  // of ranges
  float dot[2][4] = {};
  for (int tt = wave; tt * 16 < r; tt += 4) {
    const int j = tt * 16 + l16;
    f32x4 u[2] = {};
    for (int k0 = 0; k0 < r; k0 += 32) {
      const int k = k0 + 8 * g;
      const bool in = k < r && j < r;
      const V8 hi = __builtin_bit_cast(V8, in ? *reinterpret_cast<const Chunk*>(ghi + j * r + k) : zero_chunk());
      const V8 lo = __builtin_bit_cast(V8, in ? *reinterpret_cast<const Chunk*>(glo + j * r + k) : zero_chunk());
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t c = c0 + 8 * (l16 >> 2) + 4 * h + (l16 & 3);  // row l16 is register l16 % 4 of group l16 / 4
        const V8 b = __builtin_bit_cast(
            V8, k < r && c < a.out ? *reinterpret_cast<const Chunk*>(B + c * r + k) : zero_chunk());
        u[h] = Dt<DT>::mfma16(b, lo, Dt<DT>::mfma16(b, hi, u[h]));
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4* p = reinterpret_cast<const f32x4*>(a.part) + entry_of(a, rt, tt, h) * 64 + lane;
      f32x4 v = p[0];
      for (int s = 1; s < a.nSplit; ++s) v += p[s * stride];
      u[h] += v;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t c = c0 + 8 * g + 4 * h + q;
        if (j < r && c < a.out) dot[h][q] = __builtin_fmaf(static_cast<float>(B[c * r + j]), u[h][q], dot[h][q]);
      }
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float v = dot[h][q];
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
      if (l16 == 0) red[wave][8 * g + 4 * h + q] = v;
    }
  __syncthreads();
  const int64_t c = c0 + threadIdx.x;
  if (threadIdx.x < 32 && c < a.out) {
    const int t = threadIdx.x;
    const double sum = (static_cast<double>(red[0][t]) + red[1][t]) + (static_cast<double>(red[2][t]) + red[3][t]);
    const double n2 = static_cast<double>(a.base_sq[c]) + 2.0 * static_cast<double>(a.s) * sum;
    a.norm[c] = static_cast<float>(n2 > 0.0 ? sqrt(n2) : 0.0);
  }
}

}  // namespace

hipError_t launch_q4_norm_join(const Q4NormArgs& n, const Q4Parts& parts) {
  const JoinArgs a{n, parts};
  const dim3 grid(static_cast<unsigned>(q4_ceil(n.out, 32)));
  if (n.dtype == 0)
    hipLaunchKernelGGL(q4_norm_join<0>, grid, dim3(256), 0, n.stream, a);
  else
    hipLaunchKernelGGL(q4_norm_join<1>, grid, dim3(256), 0, n.stream, a);
  return hipGetLastError();
}

}  // namespace dora
