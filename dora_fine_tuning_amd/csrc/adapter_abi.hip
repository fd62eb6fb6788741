// C ABI of the operators that sort tokens by adapter and exchange rows: argument
// validation and launch.  Every check runs before the first HIP call, so invalid
// calls touch no device.
#include "../../include/dora.h"
#include "abi_common.hpp"
#include "adapter_kernels.hpp"

using namespace dora::abi;

namespace {

// Slots are numbered in 32 bits, the complement of a number included.
constexpr int64_t kMaxSlots = INT32_MAX;
constexpr int64_t kMaxCols = int64_t(1) << 22;

int check_slots(const char* fn, int64_t T, int64_t k) {
  if (T < 0 || k < 0) return fail(DORA_INVALID_ARG, "%s: negative size (%lld, %lld)", fn, (long long)T, (long long)k);
  if (T > kMaxSlots || k > kMaxSlots || T * k > kMaxSlots)
    return fail(DORA_UNSUPPORTED, "%s: %lld tokens of %lld slots are more than 2^31 - 1", fn, (long long)T,
                (long long)k);
  return DORA_OK;
}

int check_rows(const char* fn, int64_t T, int64_t k, int64_t D, int dtype) {
  if (!valid_dtype(dtype)) return fail(DORA_UNSUPPORTED, "%s: unknown dtype %d", fn, dtype);
  if (int st = check_slots(fn, T, k)) return st;
  if (D < 0) return fail(DORA_INVALID_ARG, "%s: negative size %lld", fn, (long long)D);
  if (D > kMaxCols) return fail(DORA_UNSUPPORTED, "%s: D=%lld beyond 2^22", fn, (long long)D);
  if (dora::adapter_rows_grid(T, D) * dora::kAdapterRowThreads > UINT32_MAX)
    return fail(DORA_UNSUPPORTED, "%s: T=%lld D=%lld needs more threads than one launch holds (2^32 - 1)", fn,
                (long long)T, (long long)D);
  return DORA_OK;
}

size_t mat16(int64_t rows, int64_t cols) { return static_cast<size_t>(rows) * cols * 2; }
size_t vec32(int64_t n) { return static_cast<size_t>(n) * 4; }

int need(const char* fn, const char* what, const void* p, uintptr_t align) {
  if (!p) return fail(DORA_INVALID_ARG, "%s: %s is NULL", fn, what);
  if (!aligned(p, align)) return fail(DORA_INVALID_ARG, "%s: %s needs %d-byte alignment", fn, what, (int)align);
  return DORA_OK;
}

// 16-byte rows: the sizes allow them, and so does every matrix that is there.
template <class... P>
bool wide(int64_t D, P... p) {
  return D % 8 == 0 && (... && aligned16(p));
}

}  // namespace

extern "C" {

size_t dora_adapter_sort_workspace_bytes(int64_t T, int64_t k, int64_t n) {
  if (T <= 0 || k <= 0 || n < 0 || n > dora::kMaxAdapters) return 0;
  if (T > kMaxSlots || k > kMaxSlots || T * k > kMaxSlots) return 0;
  return dora::adapter_sort_workspace_bytes(T * k, n);
}

int dora_adapter_sort(const void* ids, int id_bytes, int64_t T, int64_t k, int64_t n, int32_t* order, int32_t* place,
                      int32_t* bounds, void* ws, size_t ws_bytes, hipStream_t stream) {
  const char* fn = "dora_adapter_sort";
  if (id_bytes != 4 && id_bytes != 8) return fail(DORA_UNSUPPORTED, "%s: ids of %d bytes", fn, id_bytes);
  if (int st = check_slots(fn, T, k)) return st;
  if (n < 0) return fail(DORA_INVALID_ARG, "%s: %lld adapters", fn, (long long)n);
  if (n > dora::kMaxAdapters)
    return fail(DORA_UNSUPPORTED, "%s: %lld adapters are more than %lld", fn, (long long)n,
                (long long)dora::kMaxAdapters);
  const int64_t N = T * k;
  if (int st = need(fn, "bounds", bounds, 4)) return st;
  if (N > 0) {
    if (int st = need(fn, "ids", ids, id_bytes)) return st;
    if (int st = need(fn, "order", order, 4)) return st;
    if (int st = need(fn, "place", place, 4)) return st;
  }
  const size_t bytes = dora_adapter_sort_workspace_bytes(T, k, n);
  if (ws_bytes < bytes) return fail(DORA_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes, bytes);
  if (bytes > 0)
    if (int st = need(fn, "the workspace", ws, 16)) return st;
  const Range outs[4] = {{order, vec32(N)}, {place, vec32(N)}, {bounds, vec32(n + 1)}, {ws, bytes}};
  const Range ins[1] = {{ids, static_cast<size_t>(N) * id_bytes}};
  if (outputs_overlap(outs, ins)) return fail(DORA_INVALID_ARG, "%s: an output overlaps another argument", fn);
  const dora::AdapterSortArgs a{ids, id_bytes, N, n, order, place, bounds, ws, stream};
  return hip_status(dora::launch_adapter_sort(a), fn);
}

int dora_adapter_gather(const void* x, const int32_t* place, int64_t T, int64_t k, int64_t D, int dtype, void* rows,
                        hipStream_t stream) {
  const char* fn = "dora_adapter_gather";
  if (int st = check_rows(fn, T, k, D, dtype)) return st;
  if (T == 0 || k == 0 || D == 0) return ok();
  if (int st = need(fn, "x", x, 2)) return st;
  if (int st = need(fn, "place", place, 4)) return st;
  if (int st = need(fn, "rows", rows, 2)) return st;
  const Range outs[1] = {{rows, mat16(T * k, D)}};
  const Range ins[2] = {{x, mat16(T, D)}, {place, vec32(T * k)}};
  if (outputs_overlap(outs, ins)) return fail(DORA_INVALID_ARG, "%s: the output overlaps an input", fn);
  dora::AdapterRowsArgs a{};
  a.x = x, a.place = place, a.y = rows;
  a.T = T, a.k = k, a.D = D, a.dtype = dtype, a.vec = wide(D, x, rows), a.stream = stream;
  return hip_status(dora::launch_adapter_gather(a), fn);
}

int dora_adapter_combine(const void* rows, const float* weights, const int32_t* place, const void* base, int64_t T,
                         int64_t k, int64_t D, int dtype, void* y, hipStream_t stream) {
  const char* fn = "dora_adapter_combine";
  if (int st = check_rows(fn, T, k, D, dtype)) return st;
  if (T == 0 || D == 0) return ok();
  if (k > 0) {
    if (int st = need(fn, "rows", rows, 2)) return st;
    if (int st = need(fn, "place", place, 4)) return st;
  }
  if (!aligned(weights, 4)) return fail(DORA_INVALID_ARG, "%s: weights need 4-byte alignment", fn);
  if (!aligned(base, 2)) return fail(DORA_INVALID_ARG, "%s: base needs 2-byte alignment", fn);
  if (int st = need(fn, "y", y, 2)) return st;
  const Range outs[1] = {{y, mat16(T, D)}};
  const Range ins[3] = {{rows, mat16(T * k, D)}, {weights, vec32(T * k)}, {place, vec32(T * k)}};
  if (outputs_overlap(outs, ins) || partial_overlap(y, mat16(T, D), base, mat16(T, D)))
    return fail(DORA_INVALID_ARG, "%s: the output overlaps an input", fn);
  dora::AdapterRowsArgs a{};
  a.rows = rows, a.weights = weights, a.place = place, a.base = base, a.y = y;
  a.T = T, a.k = k, a.D = D, a.dtype = dtype, a.vec = wide(D, rows, base, y), a.stream = stream;
  return hip_status(dora::launch_adapter_combine(a), fn);
}

int dora_adapter_combine_bwd(const void* dy, const void* rows, const float* weights, const int32_t* place, int64_t T,
                             int64_t k, int64_t D, int dtype, void* d_rows, float* d_weights, hipStream_t stream) {
  const char* fn = "dora_adapter_combine_bwd";
  if (int st = check_rows(fn, T, k, D, dtype)) return st;
  if (T == 0 || k == 0 || (!d_rows && !d_weights)) return ok();
  if (D > 0) {
    if (int st = need(fn, "dy", dy, 2)) return st;
    if (d_weights)
      if (int st = need(fn, "rows", rows, 2)) return st;
  }
  if (int st = need(fn, "place", place, 4)) return st;
  if (!aligned(weights, 4) || !aligned(d_weights, 4))
    return fail(DORA_INVALID_ARG, "%s: weights and d_weights need 4-byte alignment", fn);
  if (!aligned(d_rows, 2)) return fail(DORA_INVALID_ARG, "%s: d_rows needs 2-byte alignment", fn);
  const Range outs[2] = {{d_rows, mat16(T * k, D)}, {d_weights, vec32(T * k)}};
  const Range ins[4] = {{dy, mat16(T, D)}, {rows, d_weights ? mat16(T * k, D) : 0}, {weights, vec32(T * k)},
                        {place, vec32(T * k)}};
  if (outputs_overlap(outs, ins)) return fail(DORA_INVALID_ARG, "%s: an output overlaps another argument", fn);
  dora::AdapterRowsArgs a{};
  a.x = dy, a.rows = rows, a.weights = weights, a.place = place, a.d_rows = d_rows, a.d_weights = d_weights;
  a.T = T, a.k = k, a.D = D, a.dtype = dtype, a.vec = wide(D, dy, d_weights ? rows : nullptr, d_rows);
  a.stream = stream;
  return hip_status(dora::launch_adapter_combine_bwd(a), fn);
}

}  // extern "C"
