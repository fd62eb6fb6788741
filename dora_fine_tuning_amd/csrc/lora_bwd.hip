// Backward of the compose with the adapter's second projection fused in, for
// gfx950 (press summary of arXiv:2603.22276: the training tier runs a fused
// backward; its gains come from fewer memory accesses).  With lora = h B^T
// never stored, and L = sum(dy * y):
//
//   d_base = (g - 1) * dy  (g * dy with add_base)
//   d_B    = (g * s * dy)^T h = g * s * E,            E = dy^T h   [out x r]
//   d_mag  = (sum_t dy * base + s * sum_k B * E) / n      (sum_t dy lora = sum_k B E)
//
// so neither lora nor d_lora = g * s * dy is ever formed.
//
// Kernels:
//   lora_bwd_dma      one pass over dy and base.  A workgroup owns 128 output
//                     columns x a block of rank columns x a slice of the tokens.
//                     K stages of 32 tokens: the dy rows (X panel) and h rows
//                     (Y panel) go global -> LDS by DMA, and MFMA 32x32x16
//                     contracts over the tokens, its fragments read with the
//                     transposing LDS read (ds_read_b64_tr_b16, two per
//                     fragment).  The base rows matching the dy rows come in
//                     as a third panel of the same stage, so the stage's dy
//                     and base give d_base and the column sums of dy * base.
//                     Eight tile waves run the fragment reads, the MFMAs and
//                     the elementwise part; four DMA waves issue the loads.
//                     The epilogue forms sum_k B E over its rank block and
//                     writes its E slice and its column partials.  The same
//                     kernel without the base panel is the plain contraction
//                     X^T Y over the rows of X and Y, optionally with two Y
//                     column blocks (a hi/lo pair) adding into one accumulator;
//   lora_bwd_finalize  d_mag from the partials (fp64) and d_B = g * s * (sum
//                      of the E slices), both in a fixed order, one launch;
//   lora_bwd_general  (general path) one thread per output column, all sums in
//                     order in fp32, lora per element by its r-term dot product.
#include <algorithm>
#include <type_traits>

#include "bwd_tile.hpp"
#include "lora_compose_kernels.hpp"

namespace dora {

namespace {

// One launch finishes both outputs: d_mag_j = (sum of the column partials) /
// n_j in fp64, and d_B[j][k] = (g_j * s) * (sum of the E slices, added in
// order in fp32), four elements of a row per thread and step (r % 8 == 0).
template <int DT>
__global__ __launch_bounds__(256) void lora_bwd_finalize(const float* col_part, int parts, const float* e_part,
                                                         int nSplit, int64_t out, int64_t r, const float* mag,
                                                         const float* norm, float s, float* d_mag, void* d_B) {
  using T16 = typename Dt<DT>::T;
  using T4 = T16 __attribute__((ext_vector_type(4)));
  const int64_t g0 = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t j = g0; j < out; j += stride) {
    double sum = 0.0;
    for (int p = 0; p < parts; ++p) sum += static_cast<double>(col_part[static_cast<int64_t>(p) * out + j]);
    d_mag[j] = static_cast<float>(sum / static_cast<double>(norm[j]));
  }
  const int64_t n = out * r, n4 = n / 4;
  for (int64_t e = g0; e < n4; e += stride) {
    f32x4 sum = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int p = 0; p < nSplit; ++p) sum += reinterpret_cast<const f32x4*>(e_part + static_cast<int64_t>(p) * n)[e];
    const int64_t j = (e * 4) / r;
    const float gs = (mag[j] / norm[j]) * s;
    T4 o;
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = Dt<DT>::from_f(gs * sum[q]);
    reinterpret_cast<T4*>(d_B)[e] = o;
  }
}

// General path: thread j owns output column j; everything in order in fp32.
template <int DT>
__global__ __launch_bounds__(256) void lora_bwd_general(BwdArgs a, void* d_B, float* d_mag) {
  using T16 = typename Dt<DT>::T;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (j >= a.out) return;
  const T16* dy = static_cast<const T16*>(a.dy);
  const T16* base = static_cast<const T16*>(a.base);
  const T16* h = static_cast<const T16*>(a.h);
  const T16* B = static_cast<const T16*>(a.B);
  T16* db = static_cast<T16*>(a.d_base);
  const float m = a.mag[j], n = a.norm[j];
  const float gb = a.add_base ? m / n : (m - n) / n, gs = (m / n) * a.s;
  float dm = 0.0f;
  for (int64_t t = 0; t < a.T; ++t) {
    const float d = Dt<DT>::to_f(dy[t * a.out + j]);
    float l = 0.0f;
    for (int64_t k = 0; k < a.r; ++k) l = __builtin_fmaf(Dt<DT>::to_f(h[t * a.r + k]), Dt<DT>::to_f(B[j * a.r + k]), l);
    dm = __builtin_fmaf(d, Dt<DT>::to_f(base[t * a.out + j]) + a.s * l, dm);
    if (db) db[t * a.out + j] = Dt<DT>::from_f(gb * d);
  }
  d_mag[j] = dm / n;
  for (int64_t k = 0; k < a.r; ++k) {
    float e = 0.0f;
    for (int64_t t = 0; t < a.T; ++t) e = __builtin_fmaf(Dt<DT>::to_f(dy[t * a.out + j]), Dt<DT>::to_f(h[t * a.r + k]), e);
    static_cast<T16*>(d_B)[j * a.r + k] = Dt<DT>::from_f(gs * e);
  }
}

}  // namespace

size_t lora_bwd_workspace_bytes(int64_t T, int64_t out, int64_t r) {
  if (T <= 0 || out <= 0) return 0;
  return bwd_plan(T, out, r, true).bytes;
}

int64_t lora_bwd_max_grid(int64_t T, int64_t out, int64_t r, bool vec) {
  if (!vec) return bcdiv(out, 256);
  const BwdPlan p = bwd_plan(T, out, r, true);
  return std::max<int64_t>(bcdiv(static_cast<int64_t>(p.nCB) * p.nTiles * p.nSplit, 8) * 8, bcdiv(out, 256));
}

int64_t lora_bwd_max_slice_bytes(int64_t T, int64_t out, int64_t r) {
  const BwdPlan p = bwd_plan(T, out, r, true);
  const int64_t rows = bcdiv(T, p.nSplit);
  return rows * std::max<int64_t>(out, r) * 2;
}

RowContractPlan row_contract_plan(int64_t T, int64_t nx, int64_t ny, int64_t T2, int64_t ldy) {
  RowContractPlan q;
  if (T <= 0 || nx <= 0 || ny <= 0) return q;
  const BwdPlan p = bwd_plan(T, nx, ny, true);
  q.nSplit = p.nSplit;
  q.bytes = static_cast<size_t>(q.nSplit) * nx * ny * 4;
  q.grid = bcdiv(static_cast<int64_t>(p.nCB) * p.nTiles * q.nSplit, 8) * 8;
  q.slice_bytes = bcdiv(std::max(T, T2), p.nSplit) * std::max(nx, std::max(ny, ldy)) * 2;
  return q;
}

hipError_t launch_row_contract(const void* X, const void* Y, int64_t T, int64_t nx, int64_t ny, int64_t ldy, bool dual,
                               int dtype, float* e_part, hipStream_t stream, const void* X2, const void* Y2,
                               int64_t T2) {
  if (T <= 0 || nx <= 0 || ny <= 0) return hipSuccess;
  const BwdPlan plan = bwd_plan(T, nx, ny, true);
  BwdArgs a{};
  a.dy = X;
  a.h = Y;
  a.T = T;
  a.out = nx;
  a.ldx = nx;
  a.r = ny;
  a.ldy = ldy;
  a.nCB = plan.nCB;
  a.nTiles = plan.nTiles;
  a.nSplit = plan.nSplit;
  a.e_part = e_part;
  if (T2 > 0) {
    a.dy2 = X2;
    a.h2 = Y2;
    a.T2 = T2;
  }
  auto go = [&](auto dt, auto du) {
    constexpr int DT = decltype(dt)::value;
    constexpr bool DU = decltype(du)::value;
    switch (plan.tn) {
      case 1: launch_bwd_dma<DT, 1, false, DU>(a, stream); break;
      case 2: launch_bwd_dma<DT, 2, false, DU>(a, stream); break;
      default: launch_bwd_dma<DT, 3, false, DU>(a, stream); break;
    }
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using BF = std::false_type;
  using BT = std::true_type;
  if (dtype == 0)
    dual ? go(I0{}, BT{}) : go(I0{}, BF{});
  else
    dual ? go(I1{}, BT{}) : go(I1{}, BF{});
  return hipGetLastError();
}

hipError_t launch_lora_bwd(const LoraBwdArgs& p, bool vec) {
  BwdArgs a{};
  a.dy = p.dy;
  a.base = p.base;
  a.h = p.h;
  a.B = p.B;
  a.mag = p.mag;
  a.norm = p.norm;
  a.d_base = p.d_base;
  a.s = p.s;
  a.add_base = p.add_base;
  a.T = p.T;
  a.out = p.out;
  a.r = p.r;
  a.ldx = p.out;
  a.ldy = p.r;
  if (!vec) {
    const dim3 grid(static_cast<unsigned>(bcdiv(p.out, 256)));
    if (p.dtype == 0)
      hipLaunchKernelGGL((lora_bwd_general<0>), grid, dim3(256), 0, p.stream, a, p.d_B, p.d_mag);
    else
      hipLaunchKernelGGL((lora_bwd_general<1>), grid, dim3(256), 0, p.stream, a, p.d_B, p.d_mag);
    return hipGetLastError();
  }
  const BwdPlan plan = bwd_plan(p.T, p.out, p.r, true);
  char* ws = static_cast<char*>(p.ws);
  a.nCB = plan.nCB;
  a.nTiles = plan.nTiles;
  a.nSplit = plan.nSplit;
  a.e_part = reinterpret_cast<float*>(ws);
  a.col_part = reinterpret_cast<float*>(ws + plan.off_col);
  if (p.dtype == 0) {
    switch (plan.tn) {
      case 1: launch_bwd_dma<0, 1>(a, p.stream); break;
      case 2: launch_bwd_dma<0, 2>(a, p.stream); break;
      default: launch_bwd_dma<0, 3>(a, p.stream); break;
    }
  } else {
    switch (plan.tn) {
      case 1: launch_bwd_dma<1, 1>(a, p.stream); break;
      case 2: launch_bwd_dma<1, 2>(a, p.stream); break;
      default: launch_bwd_dma<1, 3>(a, p.stream); break;
    }
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  {
    // the fast path has r >= 8, so both outputs are non-empty
    const int64_t blocks = std::min<int64_t>(bcdiv(std::max<int64_t>(p.out * p.r / 4, p.out), 256), 4096);
    if (p.dtype == 0)
      hipLaunchKernelGGL((lora_bwd_finalize<0>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0, p.stream,
                         a.col_part, plan.nSplit * plan.nTiles, a.e_part, plan.nSplit, p.out, p.r, p.mag, p.norm,
                         p.s, p.d_mag, p.d_B);
    else
      hipLaunchKernelGGL((lora_bwd_finalize<1>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0, p.stream,
                         a.col_part, plan.nSplit * plan.nTiles, a.e_part, plan.nSplit, p.out, p.r, p.mag, p.norm,
                         p.s, p.d_mag, p.d_B);
  }
  return hipGetLastError();
}

}  // namespace dora
