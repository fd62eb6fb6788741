// Backward from 8-bit checkpoints, for gfx950: the compose's backward with the
// base in 8-bit blocks, and the gradient of A from x in 8-bit blocks.
//
//   d_base = (g - 1) * dy  (g * dy with add_base), in 16 bits or packed again
//   d_B    = g * s * E,   E = dy^T h                       [out x r]
//   d_mag  = (sum_t dy * base + s * sum_k B * E) / n
//   d_A    = d_h^T x = (x^T d_h)^T                         [r x in]
//
// Both are row contractions of the tile kernel of bwd_tile.hpp; only how a panel
// comes in differs.  The compose's backward is bound by HBM: dy at 2 bytes and
// the base at 1 in, d_base at 2 or (packed) 1 out.  A workgroup's 128 columns
// are one block of every row, so the packed d_base needs no other workgroup's
// values, and the product that consumes it (dx = d_base W0) reads half the
// bytes.  The gradient of A reads x at 1 byte and is bound by the matrix pipe
// and the LDS reads that feed it.
//
// Row lengths that are not multiples of 8 (out of dy, r of h, B and d_h) are
// copied into the workspace with rows padded by zeros first: a copy of the
// operand costs less than any path of the kernel without 16-byte loads.
#include <algorithm>
#include <type_traits>

#include "bwd_tile.hpp"
#include "q8_common.hpp"

namespace dora {

namespace {

inline size_t al256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
inline int64_t up8(int64_t n) { return (n + 7) / 8 * 8; }

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

struct Q8BwdPlan {
  BwdPlan tile;
  int64_t xp = 0, rp = 0;  // padded row lengths of dy (or d_h's rank) in elements
  size_t off_dy = 0, off_h = 0, off_B = 0, bytes = 0;
  bool pad_x = false, pad_r = false;
};

// nx: columns of the X operand (out, or in); with_x: X is 16 bits (dy).
Q8BwdPlan q8_bwd_plan(int64_t T, int64_t nx, int64_t r, bool compose) {
  Q8BwdPlan p;
  p.rp = std::max<int64_t>(8, up8(r));
  p.xp = up8(nx);
  p.pad_x = compose && p.xp != nx;
  p.pad_r = p.rp != r;
  p.tile = bwd_plan(T, nx, p.rp, true);
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

template <int DT, bool BASE, int KIND>
void launch_kind(const BwdArgs& a, int tn, hipStream_t stream) {
  switch (tn) {
    case 1: launch_bwd_dma<DT, 1, BASE, false, KIND>(a, stream); break;
    case 2: launch_bwd_dma<DT, 2, BASE, false, KIND>(a, stream); break;
    default: launch_bwd_dma<DT, 3, BASE, false, KIND>(a, stream); break;
  }
}

}  // namespace

Q8BwdSizes q8_bwd_sizes(int64_t T, int64_t nx, int64_t r, bool compose) {
  const Q8BwdPlan p = q8_bwd_plan(T, nx, r, compose);
  Q8BwdSizes s;
  s.bytes = p.bytes;
  s.grid = std::max<int64_t>(static_cast<int64_t>(p.tile.nCB) * p.tile.nTiles * p.tile.nSplit + 8, q8_ceil(p.rp, 64));
  s.slice_bytes = q8_ceil(T, p.tile.nSplit) * std::max(p.xp, p.rp) * 2;
  return s;
}

hipError_t launch_q8_compose_bwd(const Q8ComposeBwdArgs& p) {
  const Q8BwdPlan plan = q8_bwd_plan(p.T, p.out, p.r, true);
  char* ws = static_cast<char*>(p.ws);
  BwdArgs a{};
  a.dy = p.dy;
  a.h = p.h;
  a.B = p.B;
  if (plan.pad_x) {
    launch_pad(p.dy, p.T, p.out, plan.xp, ws + plan.off_dy, p.stream);
    a.dy = ws + plan.off_dy;
  }
  if (plan.pad_r) {
    launch_pad(p.h, p.T, p.r, plan.rp, ws + plan.off_h, p.stream);
    launch_pad(p.B, p.out, p.r, plan.rp, ws + plan.off_B, p.stream);
    a.h = ws + plan.off_h;
    a.B = ws + plan.off_B;
  }
  a.mag = p.mag;
  a.norm = p.norm;
  a.d_base = p.d_base;
  a.s = p.s;
  a.add_base = p.add_base;
  a.T = p.T;
  a.out = p.out;
  a.r = plan.rp;
  a.ldx = plan.xp;
  a.ldy = plan.rp;
  a.nCB = plan.tile.nCB;
  a.nTiles = plan.tile.nTiles;
  a.nSplit = plan.tile.nSplit;
  a.e_part = reinterpret_cast<float*>(ws);
  a.col_part = reinterpret_cast<float*>(ws + plan.tile.off_col);
  a.q8 = static_cast<const uint8_t*>(p.bq);
  a.e8 = static_cast<const uint8_t*>(p.be);
  a.qp = q8_row_bytes(p.out);
  a.ep = q8_exp_bytes(p.out);
  a.dq8 = static_cast<uint8_t*>(p.dq);
  a.de8 = static_cast<uint8_t*>(p.de);
  if (p.T > 0) {
    if (p.dtype == 0)
      launch_kind<0, true, kBwdBase8>(a, plan.tile.tn, p.stream);
    else
      launch_kind<1, true, kBwdBase8>(a, plan.tile.tn, p.stream);
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
  BwdArgs a{};
  a.h = p.dh;
  if (plan.pad_r) {
    launch_pad(p.dh, p.T, p.r, plan.rp, ws + plan.off_h, p.stream);
    a.h = ws + plan.off_h;
  }
  a.T = p.T;
  a.out = p.in;
  a.r = plan.rp;
  a.ldx = plan.xp;
  a.ldy = plan.rp;
  a.nCB = plan.tile.nCB;
  a.nTiles = plan.tile.nTiles;
  a.nSplit = plan.tile.nSplit;
  a.e_part = reinterpret_cast<float*>(ws);
  a.q8 = static_cast<const uint8_t*>(p.xq);
  a.e8 = static_cast<const uint8_t*>(p.xe);
  a.qp = q8_row_bytes(p.in);
  a.ep = q8_exp_bytes(p.in);
  if (p.T > 0) {
    if (p.dtype == 0)
      launch_kind<0, false, kBwdX8>(a, plan.tile.tn, p.stream);
    else
      launch_kind<1, false, kBwdX8>(a, plan.tile.tn, p.stream);
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
