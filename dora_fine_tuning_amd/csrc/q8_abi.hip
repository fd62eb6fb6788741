// C ABI of the 8-bit operators: argument validation, workspace queries, launch.
// Every check runs before the first HIP call, so invalid calls touch no device.
#include "../../include/dora.h"
#include "abi_common.hpp"
#include "q8_common.hpp"

using namespace dora::abi;

namespace {

// Sizes up to here keep every product of two of them, and every byte count,
// inside 63 bits; a packed row stays below 2^22 bytes, so that 256 rows of it (or
// of 16-bit outputs) lie inside one buffer resource, and a weight's blocks are
// numbered in 30 bits.
constexpr int64_t kMaxRows = int64_t(1) << 31;
constexpr int64_t kMaxCols = (int64_t(1) << 22) - 128;
constexpr int64_t kMaxRank = int64_t(1) << 20;

int check_sizes(const char* fn, int dtype, int64_t rows, int64_t a, int64_t b) {
  if (!valid_dtype(dtype)) return fail(DORA_UNSUPPORTED, "%s: unknown dtype %d", fn, dtype);
  if (rows < 0 || a < 0 || b < 0)
    return fail(DORA_INVALID_ARG, "%s: negative size (%lld, %lld, %lld)", fn, (long long)rows, (long long)a,
                (long long)b);
  if (rows >= kMaxRows || a > kMaxCols || b > kMaxCols)
    return fail(DORA_UNSUPPORTED, "%s: sizes (%lld, %lld, %lld) beyond 2^31 rows or 2^22 columns", fn,
                (long long)rows, (long long)a, (long long)b);
  return DORA_OK;
}

size_t mat16(int64_t rows, int64_t cols) { return static_cast<size_t>(rows) * cols * 2; }
size_t row_q(int64_t rows, int64_t cols) { return static_cast<size_t>(rows) * dora::q8_row_bytes(cols); }
size_t row_e(int64_t rows, int64_t cols) { return static_cast<size_t>(rows) * dora::q8_exp_bytes(cols); }
size_t tile_q(int64_t out, int64_t in) { return row_q(dora::q8_row_bytes(out), in); }
size_t tile_e(int64_t out, int64_t in) { return row_e(dora::q8_ceil(out, dora::kQ8Block), in); }

int packed_ptrs(const char* fn, const char* what, const void* q, const void* e) {
  if (!q || !e) return fail(DORA_INVALID_ARG, "%s: %s or its exponents are NULL", fn, what);
  if (!aligned16(q) || !aligned(e, 4))
    return fail(DORA_INVALID_ARG, "%s: %s needs 16-byte alignment, its exponents 4-byte", fn, what);
  return DORA_OK;
}

// Rows of blocks of a matrix, at most 2^31 - 1 (32-bit block numbers in the kernels).
int check_blocks(const char* fn, int64_t rows, int64_t cols) {
  if (rows * dora::q8_ceil(cols, dora::kQ8Block) > INT32_MAX)
    return fail(DORA_UNSUPPORTED, "%s: %lld x %lld has more blocks than one launch holds", fn, (long long)rows,
                (long long)cols);
  return DORA_OK;
}

int pack_call(const char* fn, const void* x, int64_t rows, int64_t cols, int dtype, bool tiles, void* q, void* e,
              hipStream_t stream) {
  if (int st = check_sizes(fn, dtype, rows, cols, 0)) return st;
  if (tiles && rows > kMaxCols)
    return fail(DORA_UNSUPPORTED, "%s: out=%lld beyond 2^22", fn, (long long)rows);
  if (rows == 0 || cols == 0) return ok();
  if (!x) return fail(DORA_INVALID_ARG, "%s: the input is NULL", fn);
  if (int st = packed_ptrs(fn, "the packed output", q, e)) return st;
  if (int st = check_blocks(fn, rows, cols)) return st;
  const Range outs[2] = {{q, tiles ? tile_q(rows, cols) : row_q(rows, cols)},
                         {e, tiles ? tile_e(rows, cols) : row_e(rows, cols)}};
  const Range ins[1] = {{x, mat16(rows, cols)}};
  if (outputs_overlap(outs, ins)) return fail(DORA_INVALID_ARG, "%s: an output overlaps another argument", fn);
  const bool vec = cols % 8 == 0 && aligned16(x);
  return hip_status(tiles ? dora::launch_q8_pack_tiles(x, rows, cols, dtype, vec, q, e, stream)
                          : dora::launch_q8_pack(x, rows, cols, dtype, vec, q, e, stream),
                    fn);
}

int gemm_call(const char* fn, const void* xq, const void* xe, const void* wq, const void* we, int64_t T, int64_t out,
              int64_t in, int dtype, bool trans, void* y, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (int st = check_sizes(fn, dtype, T, out, in)) return st;
  const int64_t N = trans ? in : out, K = trans ? out : in;
  if (T == 0 || N == 0) return ok();
  if (!y) return fail(DORA_INVALID_ARG, "%s: the output is NULL", fn);
  if (!aligned(y, 2)) return fail(DORA_INVALID_ARG, "%s: the output needs 2-byte alignment", fn);
  if (K > 0) {
    if (int st = packed_ptrs(fn, "the packed rows", xq, xe)) return st;
    if (int st = packed_ptrs(fn, "the packed weight", wq, we)) return st;
  }
  const size_t need = dora::q8_gemm_workspace_bytes(T, out, in, trans);
  if (ws_bytes < need) return fail(DORA_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes, need);
  if (need > 0 && (!ws || !aligned16(ws)))
    return fail(DORA_INVALID_ARG, "%s: workspace is NULL or not 16-byte aligned", fn);
  const Range outs[2] = {{y, mat16(T, N)}, {ws, need}};
  const Range ins[4] = {{xq, row_q(T, K)}, {xe, row_e(T, K)}, {wq, tile_q(out, in)}, {we, tile_e(out, in)}};
  if (outputs_overlap(outs, ins)) return fail(DORA_INVALID_ARG, "%s: an output overlaps another argument", fn);
  if (dora::q8_gemm_max_grid(T, out, in, trans) > INT32_MAX)
    return fail(DORA_UNSUPPORTED, "%s: T=%lld out=%lld in=%lld needs more workgroups than one launch holds", fn,
                (long long)T, (long long)out, (long long)in);
  const dora::Q8GemmArgs a{xq, xe, wq, we, T, out, in, dtype, trans, y, ws, stream};
  return hip_status(dora::launch_q8_gemm(a), fn);
}

}  // namespace

extern "C" {

int dora_q8_pack(const void* x, int64_t rows, int64_t cols, int dtype, void* q, void* e, hipStream_t stream) {
  return pack_call("dora_q8_pack", x, rows, cols, dtype, false, q, e, stream);
}

int dora_q8_pack_weight(const void* W, int64_t out, int64_t in, int dtype, void* q, void* e, hipStream_t stream) {
  return pack_call("dora_q8_pack_weight", W, out, in, dtype, true, q, e, stream);
}

int dora_q8_unpack(const void* q, const void* e, int64_t rows, int64_t cols, int weight, int dtype, void* x,
                   hipStream_t stream) {
  const char* fn = "dora_q8_unpack";
  if (int st = check_sizes(fn, dtype, rows, cols, 0)) return st;
  if (rows == 0 || cols == 0) return ok();
  if (!x) return fail(DORA_INVALID_ARG, "%s: the output is NULL", fn);
  if (int st = packed_ptrs(fn, "the packed input", q, e)) return st;
  if (int st = check_blocks(fn, rows, cols)) return st;
  const Range outs[1] = {{x, mat16(rows, cols)}};
  const Range ins[2] = {{q, row_q(rows, cols)},
                        {e, weight ? row_e(dora::q8_ceil(rows, dora::kQ8Block), cols) : row_e(rows, cols)}};
  if (outputs_overlap(outs, ins)) return fail(DORA_INVALID_ARG, "%s: the output overlaps an input", fn);
  const bool vec = cols % 8 == 0 && aligned16(x);
  return hip_status(dora::launch_q8_unpack(q, e, rows, cols, weight != 0, dtype, vec, x, stream), fn);
}

size_t dora_q8_linear_workspace_bytes(int64_t T, int64_t out, int64_t in) {
  if (T <= 0 || out <= 0 || in <= 0 || T >= kMaxRows || out > kMaxCols || in > kMaxCols) return 0;
  return dora::q8_gemm_workspace_bytes(T, out, in, false);
}

int dora_q8_linear_fwd(const void* xq, const void* xe, const void* wq, const void* we, int64_t T, int64_t out,
                       int64_t in, int dtype, void* y, void* ws, size_t ws_bytes, hipStream_t stream) {
  return gemm_call("dora_q8_linear_fwd", xq, xe, wq, we, T, out, in, dtype, false, y, ws, ws_bytes, stream);
}

size_t dora_q8_linear_bwd_workspace_bytes(int64_t T, int64_t out, int64_t in) {
  if (T <= 0 || out <= 0 || in <= 0 || T >= kMaxRows || out > kMaxCols || in > kMaxCols) return 0;
  return dora::q8_gemm_workspace_bytes(T, out, in, true);
}

int dora_q8_linear_bwd(const void* gq, const void* ge, const void* wq, const void* we, int64_t T, int64_t out,
                       int64_t in, int dtype, void* dx, void* ws, size_t ws_bytes, hipStream_t stream) {
  return gemm_call("dora_q8_linear_bwd", gq, ge, wq, we, T, out, in, dtype, true, dx, ws, ws_bytes, stream);
}

size_t dora_q8_lora_compose_bwd_workspace_bytes(int64_t T, int64_t out, int64_t r) {
  if (T < 0 || out <= 0 || r < 0 || T >= kMaxRows || out > kMaxCols || r > kMaxRank) return 0;
  return dora::q8_bwd_sizes(T, out, r, true).bytes;
}

int dora_q8_lora_compose_bwd(const void* dy, const void* bq, const void* be, const void* h, const void* B,
                             const float* mag, const float* norm, float s, int64_t T, int64_t out, int64_t r,
                             int dtype, int add_base, void* d_base, void* dq, void* de, void* d_B, float* d_mag,
                             void* ws, size_t ws_bytes, hipStream_t stream) {
  const char* fn = "dora_q8_lora_compose_bwd";
  if (int st = check_sizes(fn, dtype, T, out, r)) return st;
  if (r > kMaxRank) return fail(DORA_UNSUPPORTED, "%s: r=%lld beyond 2^20", fn, (long long)r);
  if (out == 0) return ok();
  if (!mag || !norm || !d_mag) return fail(DORA_INVALID_ARG, "%s: mag, norm or d_mag is NULL", fn);
  if (T > 0) {
    if (!dy || !aligned16(dy)) return fail(DORA_INVALID_ARG, "%s: dy is NULL or not 16-byte aligned", fn);
    if (int st = packed_ptrs(fn, "the packed base", bq, be)) return st;
  }
  if (r > 0 && (!B || !d_B)) return fail(DORA_INVALID_ARG, "%s: B or d_B is NULL", fn);
  if (T > 0 && r > 0 && !h) return fail(DORA_INVALID_ARG, "%s: h is NULL", fn);
  if (!aligned16(h) || !aligned16(B) || !aligned16(d_base) || !aligned16(d_B))
    return fail(DORA_INVALID_ARG, "%s: h, B, d_base and d_B need 16-byte alignment", fn);
  if ((dq == nullptr) != (de == nullptr)) return fail(DORA_INVALID_ARG, "%s: dq and de come together", fn);
  if (dq)
    if (int st = packed_ptrs(fn, "the packed d_base", dq, de)) return st;
  const dora::Q8BwdSizes sz = dora::q8_bwd_sizes(T, out, r, true);
  if (sz.grid > INT32_MAX)
    return fail(DORA_UNSUPPORTED, "%s: T=%lld out=%lld r=%lld: more workgroups than one launch holds", fn, (long long)T,
                (long long)out, (long long)r);
  if (ws_bytes < sz.bytes) return fail(DORA_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes, sz.bytes);
  if (sz.bytes > 0 && (!ws || !aligned16(ws)))
    return fail(DORA_INVALID_ARG, "%s: workspace is NULL or not 16-byte aligned", fn);
  const size_t vb = static_cast<size_t>(out) * 4;
  const Range ins[7] = {{dy, mat16(T, out)}, {bq, row_q(T, out)}, {be, row_e(T, out)}, {h, mat16(T, r)},
                        {B, mat16(out, r)},  {mag, vb},           {norm, vb}};
  const Range outs[6] = {{d_base, mat16(T, out)}, {dq, row_q(T, out)}, {de, row_e(T, out)},
                         {d_B, mat16(out, r)},    {d_mag, vb},         {ws, sz.bytes}};
  if (outputs_overlap(outs, ins)) return fail(DORA_INVALID_ARG, "%s: an output overlaps another argument", fn);
  const dora::Q8ComposeBwdArgs a{dy, bq, be, h, B, mag, norm, s, T, out, r, dtype, add_base ? 1 : 0,
                                 d_base, dq, de, d_B, d_mag, ws, stream};
  return hip_status(dora::launch_q8_compose_bwd(a), fn);
}

size_t dora_q8_grad_a_workspace_bytes(int64_t T, int64_t in, int64_t r) {
  if (T < 0 || in <= 0 || r <= 0 || T >= kMaxRows || in > kMaxCols || r > kMaxRank) return 0;
  return dora::q8_bwd_sizes(T, in, r, false).bytes;
}

int dora_q8_grad_a(const void* dh, const void* xq, const void* xe, int64_t T, int64_t in, int64_t r, int dtype,
                   void* d_A, void* ws, size_t ws_bytes, hipStream_t stream) {
  const char* fn = "dora_q8_grad_a";
  if (int st = check_sizes(fn, dtype, T, in, r)) return st;
  if (r > kMaxRank) return fail(DORA_UNSUPPORTED, "%s: r=%lld beyond 2^20", fn, (long long)r);
  if (in == 0 || r == 0) return ok();
  if (!d_A || !aligned(d_A, 2)) return fail(DORA_INVALID_ARG, "%s: d_A is NULL or not 2-byte aligned", fn);
  if (T > 0) {
    if (!dh || !aligned16(dh)) return fail(DORA_INVALID_ARG, "%s: d_h is NULL or not 16-byte aligned", fn);
    if (int st = packed_ptrs(fn, "the packed x", xq, xe)) return st;
  }
  const dora::Q8BwdSizes sz = dora::q8_bwd_sizes(T, in, r, false);
  if (sz.grid > INT32_MAX)
    return fail(DORA_UNSUPPORTED, "%s: T=%lld in=%lld r=%lld: more workgroups than one launch holds", fn, (long long)T,
                (long long)in, (long long)r);
  if (ws_bytes < sz.bytes) return fail(DORA_INVALID_ARG, "%s: workspace of %zu bytes, %zu needed", fn, ws_bytes, sz.bytes);
  if (sz.bytes > 0 && (!ws || !aligned16(ws)))
    return fail(DORA_INVALID_ARG, "%s: workspace is NULL or not 16-byte aligned", fn);
  const Range ins[3] = {{dh, mat16(T, r)}, {xq, row_q(T, in)}, {xe, row_e(T, in)}};
  const Range outs[2] = {{d_A, mat16(r, in)}, {ws, sz.bytes}};
  if (outputs_overlap(outs, ins)) return fail(DORA_INVALID_ARG, "%s: an output overlaps another argument", fn);
  const dora::Q8GradAArgs a{dh, xq, xe, T, in, r, dtype, d_A, ws, stream};
  return hip_status(dora::launch_q8_grad_a(a), fn);
}

}  // extern "C"
