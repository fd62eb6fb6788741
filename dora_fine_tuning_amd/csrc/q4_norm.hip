// The factored norm of a 4-bit weight with a cached base term, for gfx950:
//
//   n_i = sqrt(c_i + 2 s sum_j B_ij U_ij),  U = W A^T + (s/2) B (A A^T),
//
// c_i = ||W_i||^2.  W A^T is the forward product on the r rows of A, whose fp32 sums
// stay in the workspace as its kernels leave them (q4_gemm.hip): 17/32 bytes an element
// of W are read instead of the 5 that unpacking to 16 bits, and reading that, take.
// Whole calls: 26 us at rank 16 of 8192^2 (168 by unpacked rows), 41 at rank 64 of
// 27648 x 5120 (590), 83 at rank 384 of 8192^2 (195): of these 48 the product, 27 the join
// and 12 the Gram matrix.
// (s/2) A A^T comes as two 16-bit matrices from the 16-bit norm's Gram kernels (norm.hip).
#include <algorithm>

#include "q4_common.hpp"

namespace dora {

namespace {

constexpr int kMaxWaves = 16;

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

// A workgroup 64 outputs, whose rows of B stand in LDS as fragments (KS steps of 32 of the
// rank); its waves, one for 16 rows of A and 16 at most, take 16 rows of A in turn: B times
// (s/2) A A^T by the matrix instruction, in the layout of the entries, these added in the
// order of their ranges, and the dot with B.  The loads bound it: 27 us at rank 384 of 8192
// outputs and 90 at rank 512 of 27648 (40 and 260 with B from the caches too, workgroups of
// 32 outputs; 65 and 89 with B in registers and (s/2) A A^T through LDS, in step), 10 at
// rank 64.
template <int DT, int KS>
__global__ __launch_bounds__(64 * kMaxWaves) void q4_norm_join(JoinArgs a) {
  using T16 = typename Dt<DT>::T;
  using V8 = typename Dt<DT>::V8;
  __shared__ Chunk bs[KS * 4][64];  // step, row tile, half
  __shared__ float red[kMaxWaves][64];
  const int lane = threadIdx.x & 63, l16 = lane & 15, g = lane >> 4, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t rt = 2 * static_cast<int64_t>(blockIdx.x), c0 = rt * 32;
  const int r = static_cast<int>(a.r), steps = (r + 31) / 32;
  const int tiles = c0 + 32 < a.out ? 2 : 1;
  const int64_t stride = a.all * (a.few ? a.R * a.NT * 2 : a.WM * a.WN * a.TMW * a.TNW) * 64;  // of ranges
  // eight elements of a row from 32 ks + 8 g on, zeros past its end
  auto chunk = [&](const T16* row, int ks) {
    const int k = 32 * ks + 8 * g;
    const Chunk c = *reinterpret_cast<const Chunk*>(row + min(k, r - 8));
    return k < r ? c : zero_chunk();
  };
  // Row l16 of the product's left operand comes out as register l16 % 4 of lane group
  // l16 / 4.  Rows past the last are that one again, and not used.
  for (int f = wave; f < 4 * steps; f += waves) {
    const int64_t c = c0 + 32 * ((f >> 1) & 1) + 8 * (l16 >> 2) + 4 * (f & 1) + (l16 & 3);
    bs[f][lane] = chunk(static_cast<const T16*>(a.B) + min(c, a.out - 1) * r, f >> 2);
  }
  __syncthreads();
  float dot[4][4] = {};
  for (int tt = wave; 16 * tt < r; tt += waves) {
    const int j = 16 * tt + l16, row = min(j, r - 1) * r;
    const T16 *hp = static_cast<const T16*>(a.ghi) + row, *lp = static_cast<const T16*>(a.glo) + row;
    const f32x4* p[4];
    f32x4 v[4], u[4] = {};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      p[x] = reinterpret_cast<const f32x4*>(a.part) + entry_of(a, rt + ((x >> 1) & (tiles - 1)), tt, x & 1) * 64 + lane;
      v[x] = *p[x];
    }
    for (int k0 = 0; k0 < steps; k0 += 4) {  // the loads of four steps before their products
      Chunk hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) hi[i] = chunk(hp, k0 + i), lo[i] = chunk(lp, k0 + i);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (k0 + i < steps) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const V8 w = __builtin_bit_cast(V8, bs[(k0 + i) * 4 + x][lane]);
            u[x] = Dt<DT>::mfma16(w, __builtin_bit_cast(V8, hi[i]), u[x]);
            u[x] = Dt<DT>::mfma16(w, __builtin_bit_cast(V8, lo[i]), u[x]);
          }
        }
      }
    }
    for (int s = 1; s < a.nSplit; ++s)
#pragma unroll
      for (int x = 0; x < 4; ++x) v[x] += p[x][s * stride];
    // B at output 8 g + 4 h + q and column j, of which bs has eight a lane
    const T16* bj = reinterpret_cast<const T16*>(&bs[(j >> 5) * 4][16 * ((j >> 3) & 3) + 4 * g]) + (j & 7);
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (j < r) dot[x][q] = __builtin_fmaf(static_cast<float>(bj[(x * 64 + q) * 8]), u[x][q] + v[x][q], dot[x][q]);
  }
#pragma unroll
  for (int x = 0; x < 4; ++x)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float d = dot[x][q];
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) d += __shfl_xor(d, o, 64);
      if (l16 == 0) red[wave][32 * (x >> 1) + 8 * g + 4 * (x & 1) + q] = d;
    }
  __syncthreads();
  const int64_t c = c0 + threadIdx.x;
  if (threadIdx.x < 64 && c < a.out) {
    double sum = 0.0;
    for (int w = 0; w < waves; ++w) sum += static_cast<double>(red[w][threadIdx.x]);
    const double n2 = static_cast<double>(a.base_sq[c]) + 2.0 * static_cast<double>(a.s) * sum;
    a.norm[c] = static_cast<float>(n2 > 0.0 ? sqrt(n2) : 0.0);
  }
}

template <int DT>
void launch_join(const JoinArgs& a) {
  const dim3 grid(static_cast<unsigned>(q4_ceil(a.out, 64)));
  const dim3 block(static_cast<unsigned>(64 * std::min<int64_t>(q4_ceil(a.r, 16), kMaxWaves)));
  if (a.r <= 128)  // less LDS: more workgroups a CU
    hipLaunchKernelGGL((q4_norm_join<DT, 4>), grid, block, 0, a.stream, a);
  else  // r <= 512
    hipLaunchKernelGGL((q4_norm_join<DT, 16>), grid, block, 0, a.stream, a);
}

}  // namespace

hipError_t launch_q4_norm_join(const Q4NormArgs& n, const Q4Parts& parts) {
  const JoinArgs a{n, parts};
  if (n.dtype == 0)
    launch_join<0>(a);
  else
    launch_join<1>(a);
  return hipGetLastError();
}

}  // namespace dora
