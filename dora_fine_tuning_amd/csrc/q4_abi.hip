// C ABI of the 4-bit weight: argument validation, workspace queries, launch.
// Every check runs before the first HIP call, so invalid calls touch no device.
#include <algorithm>

#include "../../include/dora.h"
#include "abi_common.hpp"
#include "norm_kernels.hpp"
#include "q4_common.hpp"

using namespace dora::abi;

namespace {

// Sizes up to here keep every product of two of them, and every byte count,
// inside 63 bits, and 256 rows of 16-bit values inside one buffer resource.
constexpr int64_t kMaxRows = int64_t(1) << 31;
constexpr int64_t kMaxCols = (int64_t(1) << 22) - 128;

int check_sizes(const char* fn, int dtype, int64_t T, int64_t out, int64_t in) {
  if (!valid_dtype(dtype)) return fail(DORA_UNSUPPORTED, "%s: unknown dtype %d", fn, dtype);
  if (T < 0 || out < 0 || in < 0)
    return fail(DORA_INVALID_ARG, "%s: negative size (%lld, %lld, %lld)", fn, (long long)T, (long long)out,
                (long long)in);
  if (T >= kMaxRows || out > kMaxCols || in > kMaxCols)
    return fail(DORA_UNSUPPORTED, "%s: sizes (%lld, %lld, %lld) beyond 2^31 rows or 2^22 columns", fn, (long long)T,
                (long long)out, (long long)in);
  if (dora::q4_ceil(out, dora::kQ4Rows) * dora::q4_ceil(in, dora::kQ4Cols) > INT32_MAX)
    return fail(DORA_UNSUPPORTED, "%s: a weight of %lld x %lld has more tiles than one launch holds", fn,
                (long long)out, (long long)in);
  return DORA_OK;
}

// Packing and unpacking: a launch holds fewer than 2^32 threads.
int check_pack(const char* fn, int dtype, int64_t out, int64_t in) {
  if (int st = check_sizes(fn, dtype, 0, out, in)) return st;
  if (dora::q4_pack_grid(out, in) * 256 > UINT32_MAX)
    return fail(DORA_UNSUPPORTED, "%s: a weight of %lld x %lld needs more threads than one launch holds", fn,
                (long long)out, (long long)in);
  return DORA_OK;
}

size_t mat16(int64_t rows, int64_t cols) { return static_cast<size_t>(rows) * cols * 2; }
size_t tiles(int64_t out, int64_t in) {
  return static_cast<size_t>(dora::q4_ceil(out, dora::kQ4Rows)) * dora::q4_ceil(in, dora::kQ4Cols);
}
size_t weight_q(int64_t out, int64_t in) { return tiles(out, in) * dora::kQ4TileQ; }
size_t weight_e(int64_t out, int64_t in) { return tiles(out, in) * dora::kQ4TileE; }

int weight_ptrs(const char* fn, const void* q, const void* e) {
  if (!q || !e) return fail(DORA_INVALID_ARG, "%s: the packed weight or its exponents are NULL", fn);
  if (!aligned16(q) || !aligned16(e))
    return fail(DORA_INVALID_ARG, "%s: the packed weight and its exponents need 16-byte alignment", fn);
  return DORA_OK;
}

// The plan of a call, which depends on its sizes alone.  Weighing the kernels takes
// 1.6 us, twice a call (workspace, product), next to 5 us of a single token's kernel:
// each thread keeps the plans of the sizes it met last.
const dora::Q4Plan& plan_of(int64_t T, int64_t out, int64_t in, bool trans) {
  struct Entry {
    int64_t T = 0, out = 0, in = 0;
    bool trans = false;
    dora::Q4Plan plan;
  };
  static thread_local Entry table[64];
  constexpr uint64_t kOdd = 0x9e3779b97f4a7c15u;
  const uint64_t mix = (static_cast<uint64_t>(T) * kOdd ^ static_cast<uint64_t>(out)) * kOdd ^
                       static_cast<uint64_t>(in) * 2 ^ (trans ? 1u : 0u);
  Entry& e = table[mix * kOdd >> 58];
  if (e.T != T || e.out != out || e.in != in || e.trans != trans)  // (T >= 1)
    e = Entry{T, out, in, trans, dora::q4_plan(T, out, in, trans)};
  return e.plan;
}

size_t workspace(int64_t T, int64_t out, int64_t in, bool trans) {
  if (T <= 0 || out <= 0 || in <= 0 || T >= kMaxRows || out > kMaxCols || in > kMaxCols) return 0;
  return plan_of(T, out, in, trans).workspace();
}

int gemm_call(const char* fn, const void* x, const void* q, const void* e, int64_t T, int64_t out, int64_t in,
              int dtype, bool trans, void* y, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (int st = check_sizes(fn, dtype, T, out, in)) return st;
  const int64_t N = trans ? in : out, K = trans ? out : in;
  if (T == 0 || N == 0) return ok();
  if (!y) return fail(DORA_INVALID_ARG, "%s: the output is NULL", fn);
  if (!aligned(y, 2)) return fail(DORA_INVALID_ARG, "%s: the output needs 2-byte alignment", fn);
  if (K > 0) {
    if (!x || !aligned16(x)) return fail(DORA_INVALID_ARG, "%s: the rows are NULL or not 16-byte aligned", fn);
    if (int st = weight_ptrs(fn, q, e)) return st;
  }
  const dora::Q4Plan& plan = plan_of(T, out, in, trans);
  const size_t need = K > 0 ? plan.workspace() : 0;
  if (ws_bytes < need) return fail(DORA_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes, need);
  if (need > 0 && (!ws || !aligned16(ws)))
    return fail(DORA_INVALID_ARG, "%s: workspace is NULL or not 16-byte aligned", fn);
  const Range outs[2] = {{y, mat16(T, N)}, {ws, need}};
  const Range ins[3] = {{x, mat16(T, K)}, {q, weight_q(out, in)}, {e, weight_e(out, in)}};
  if (outputs_overlap(outs, ins)) return fail(DORA_INVALID_ARG, "%s: an output overlaps another argument", fn);
  if (plan.units() > INT32_MAX)
    return fail(DORA_UNSUPPORTED, "%s: T=%lld out=%lld in=%lld needs more workgroups than one launch holds", fn,
                (long long)T, (long long)out, (long long)in);
  const dora::Q4GemmArgs a{x, q, e, T, out, in, dtype, trans, y, ws, stream};
  return hip_status(dora::launch_q4_gemm(a, plan), fn);
}

// The norm: ranks whose sums, fp32 [r x out], are small beside the weight in 16 bits, and
// the Gram kernels' own limit of columns.
constexpr int64_t kNormMaxRank = 512, kNormMaxCols = int64_t(1) << 21;

bool norm_takes(int64_t out, int64_t in, int64_t r) {
  return out > 0 && in > 0 && r > 0 && out <= kMaxCols && in < kNormMaxCols && r <= kNormMaxRank && in % 8 == 0 &&
         r % 8 == 0;
}
// Its workspace: the Gram kernels' (their plan), then the product's sums.
struct NormPlans {
  dora::NormPlan gram;
  dora::Q4Plan product;
  size_t at() const { return (gram.bytes + 255) / 256 * 256; }
  size_t bytes() const { return at() + product.workspace(); }
};
NormPlans norm_plans(int64_t out, int64_t in, int64_t r, int dtype) {
  return {dora::make_norm_plan(out, in, r, dtype, true), dora::q4_parts_plan(plan_of(r, out, in, false), r)};
}

}  // namespace

extern "C" {

int dora_q4_pack_weight(const void* W, int64_t out, int64_t in, int dtype, void* q, void* e, hipStream_t stream) {
  const char* fn = "dora_q4_pack_weight";
  if (int st = check_pack(fn, dtype, out, in)) return st;
  if (out == 0 || in == 0) return ok();
  if (!W || !aligned(W, 2)) return fail(DORA_INVALID_ARG, "%s: the weight is NULL or not 2-byte aligned", fn);
  if (int st = weight_ptrs(fn, q, e)) return st;
  const Range outs[2] = {{q, weight_q(out, in)}, {e, weight_e(out, in)}};
  const Range ins[1] = {{W, mat16(out, in)}};
  if (outputs_overlap(outs, ins)) return fail(DORA_INVALID_ARG, "%s: an output overlaps another argument", fn);
  return hip_status(dora::launch_q4_pack(W, out, in, dtype, in % 8 == 0 && aligned16(W), q, e, stream), fn);
}

int dora_q4_unpack_weight(const void* q, const void* e, int64_t rows, int64_t cols, int dtype, void* W,
                          hipStream_t stream) {
  const char* fn = "dora_q4_unpack_weight";
  if (int st = check_pack(fn, dtype, rows, cols)) return st;
  if (rows == 0 || cols == 0) return ok();
  if (!W || !aligned(W, 2)) return fail(DORA_INVALID_ARG, "%s: the output is NULL or not 2-byte aligned", fn);
  if (int st = weight_ptrs(fn, q, e)) return st;
  const Range outs[1] = {{W, mat16(rows, cols)}};
  const Range ins[2] = {{q, weight_q(rows, cols)}, {e, weight_e(rows, cols)}};
  if (outputs_overlap(outs, ins)) return fail(DORA_INVALID_ARG, "%s: the output overlaps an input", fn);
  return hip_status(dora::launch_q4_unpack(q, e, rows, cols, dtype, cols % 8 == 0 && aligned16(W), W, stream), fn);
}

size_t dora_q4_linear_workspace_bytes(int64_t T, int64_t out, int64_t in) { return workspace(T, out, in, false); }

int dora_q4_linear_fwd(const void* x, const void* q, const void* e, int64_t T, int64_t out, int64_t in, int dtype,
                       void* y, void* ws, size_t ws_bytes, hipStream_t stream) {
  return gemm_call("dora_q4_linear_fwd", x, q, e, T, out, in, dtype, false, y, ws, ws_bytes, stream);
}

size_t dora_q4_linear_bwd_workspace_bytes(int64_t T, int64_t out, int64_t in) { return workspace(T, out, in, true); }

int dora_q4_linear_bwd(const void* g, const void* q, const void* e, int64_t T, int64_t out, int64_t in, int dtype,
                       void* dx, void* ws, size_t ws_bytes, hipStream_t stream) {
  return gemm_call("dora_q4_linear_bwd", g, q, e, T, out, in, dtype, true, dx, ws, ws_bytes, stream);
}

int dora_q4_plan(int64_t T, int64_t out, int64_t in, int product, int64_t* plan) {
  const char* fn = "dora_q4_plan";
  if (int st = check_sizes(fn, 0, T, out, in)) return st;
  if (!plan) return fail(DORA_INVALID_ARG, "%s: plan is NULL", fn);
  if (product < 0 || product > 2) return fail(DORA_INVALID_ARG, "%s: unknown product %d", fn, product);
  if (product == 2 && out > 0 && !norm_takes(out, in, T))
    return fail(DORA_UNSUPPORTED, "%s: out=%lld in=%lld r=%lld is not taken by the norm", fn, (long long)out,
                (long long)in, (long long)T);
  std::fill(plan, plan + 6, 0);
  if (T == 0 || out == 0 || in == 0) return ok();
  dora::Q4Plan p = plan_of(T, out, in, product == 1);
  if (product == 2) p = dora::q4_parts_plan(p, T);
  dora::q4_plan_numbers(p, product == 1, plan);
  return ok();
}

size_t dora_q4_norm_workspace_bytes(int64_t out, int64_t in, int64_t r, int dtype) {
  return valid_dtype(dtype) && norm_takes(out, in, r) ? norm_plans(out, in, r, dtype).bytes() : 0;
}

int dora_q4_norm_cached(const void* q, const void* e, const void* A, const void* B, const float* base_sq, int64_t out,
                        int64_t in, int64_t r, float s, int dtype, float* norm_out, void* ws, size_t ws_bytes,
                        hipStream_t stream) {
  const char* fn = "dora_q4_norm_cached";
  if (int st = check_sizes(fn, dtype, r, out, in)) return st;
  if (out == 0) return ok();
  if (!norm_takes(out, in, r))
    return fail(DORA_UNSUPPORTED, "%s: out=%lld in=%lld r=%lld: in and r are to be multiples of 8, r up to %lld", fn,
                (long long)out, (long long)in, (long long)r, (long long)kNormMaxRank);
  if (int st = weight_ptrs(fn, q, e)) return st;
  if (!A || !B || !aligned16(A) || !aligned16(B))
    return fail(DORA_INVALID_ARG, "%s: A or B is NULL or not 16-byte aligned", fn);
  if (!base_sq || !norm_out || !aligned(base_sq, 4) || !aligned(norm_out, 4))
    return fail(DORA_INVALID_ARG, "%s: base_sq or norm_out is NULL or not 4-byte aligned", fn);
  const NormPlans p = norm_plans(out, in, r, dtype);
  if (ws_bytes < p.bytes())
    return fail(DORA_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes, p.bytes());
  if (!ws || !aligned16(ws)) return fail(DORA_INVALID_ARG, "%s: workspace is NULL or not 16-byte aligned", fn);
  const size_t n4 = static_cast<size_t>(out) * 4;
  const Range outs[2] = {{norm_out, n4}, {ws, p.bytes()}};
  const Range ins[5] = {
      {q, weight_q(out, in)}, {e, weight_e(out, in)}, {A, mat16(r, in)}, {B, mat16(out, r)}, {base_sq, n4}};
  if (outputs_overlap(outs, ins)) return fail(DORA_INVALID_ARG, "%s: an output overlaps another argument", fn);
  if (p.product.units() > INT32_MAX || dora::norm_max_grid(p.gram) > INT32_MAX)
    return fail(DORA_UNSUPPORTED, "%s: out=%lld in=%lld r=%lld needs more workgroups than one launch holds", fn,
                (long long)out, (long long)in, (long long)r);
  char* w = static_cast<char*>(ws);
  if (int st = hip_status(dora::launch_norm_gram(p.gram, A, s * 0.5f, w, stream), fn)) return st;
  const dora::Q4GemmArgs a{A, q, e, r, out, in, dtype, false, nullptr, w + p.at(), stream};
  if (int st = hip_status(dora::launch_q4_gemm(a, p.product), fn)) return st;
  const dora::Q4NormArgs n{B, w + p.gram.off_ghi, w + p.gram.off_glo, base_sq, reinterpret_cast<float*>(w + p.at()),
                           out, r, dtype, s, norm_out, stream};
  return hip_status(dora::launch_q4_norm_join(n, dora::q4_parts_of(p.product, r)), fn);
}

}  // extern "C"
