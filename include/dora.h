/*
 * dora.h -- C ABI of the DoRA adapter hot path on AMD Instinct MI355X (gfx950).
 *
 * DoRA (weight-decomposed low-rank adaptation) scales each output row of the
 * adapted weight W0 + s*B*A by g = m / n, where m is a trained magnitude and
 * n = ||W0_i + s*B_i*A||_2 is the weight norm of that row.  This library
 * provides the three operations that the press summary of arXiv:2603.22276
 * ("AI training breakthrough: Anthropic team cracks the memory bottleneck of
 * large-model fine-tuning", techwalker.com/2026/0401/3182870) singles out:
 *
 *   dora_norm_factored  the weight norm as base + cross + Gram terms, never
 *                       forming the out x in matrix B*A (paragraph on the
 *                       "factored norm");
 *   dora_compose_fwd    the fused magnitude compose in its stable form
 *                       (g-1)*base + g*s*lora with fp32 intermediates
 *                       (paragraphs on the fused kernel and on stability near
 *                       g = 1; the forward-only inference tier);
 *   dora_compose_bwd    its fused backward with the magnitude-gradient token
 *                       reduction (paragraphs on the three-tier dispatch and on
 *                       the convergence study's dmag reduction).
 *
 * and the compose with the adapter's second projection fused in, so that lora
 * is never stored (the page's account of where the fused kernel's gains come
 * from: fewer memory accesses):
 *
 *   dora_lora_compose_fwd      y = (g-1)*base + g*s*(h*B^T), h = x*A^T;
 *   dora_lora_compose_bwd      its backward: d_base, d_B and d_mag from dy,
 *                              base and h, without lora or d_lora;
 *
 * for a caller that does not treat the norm as a constant:
 *
 *   dora_norm_bwd              d_A and d_B of the weight norm, from dL/dn,
 *                              without forming B*A;
 *   dora_norm_bwd_slab         the same from a W0 in slabs of rows;
 *
 * and, for the cached base norm the page lists as future work (W0 is frozen):
 *
 *   dora_row_sqnorm            ||W0_i||^2 per row, computed once;
 *   dora_norm_factored_cached  the weight norm with that cache as its base term;
 *
 * and, for the layer's frozen side in 8 bits (W0, and what the backward needs of
 * the activations):
 *
 *   dora_q8_pack, dora_q8_pack_weight, dora_q8_unpack
 *                              blocks of 128 of e4m3 with a power-of-two scale;
 *   dora_q8_linear_fwd, dora_q8_linear_bwd
 *                              x W0^T and g W0 on packed operands;
 *   dora_q8_lora_compose_bwd   dora_lora_compose_bwd from a packed base;
 *   dora_q8_grad_a             d_A from packed x;
 *
 * and, for a frozen W0 in 4 bits:
 *
 *   dora_q4_pack_weight, dora_q4_unpack_weight
 *                              blocks of 32 of e2m1 with a power-of-two scale;
 *   dora_q4_linear_fwd, dora_q4_linear_bwd
 *                              x W0^T and g W0 with 16-bit x and g;
 *   dora_q4_norm_cached        dora_norm_factored_cached of a packed W0;
 *
 * and, for a batch whose tokens use different adapters over the one W0:
 *
 *   dora_adapter_sort          tokens' slots sorted by adapter;
 *   dora_adapter_gather        tokens' rows in that order;
 *   dora_adapter_combine       rows added up per token, with weights;
 *   dora_adapter_combine_bwd   its gradients of the rows and the weights.
 *
 * Conventions shared by every entry point
 *  - Matrices are row-major and contiguous.  W0 is [out x in], A is [r x in],
 *    B is [out x r] (nn.Linear orientation); base, lora, y, dy, d_lora and
 *    d_base are [T x out] (T tokens).  Vectors mag (m), norm (n) and d_mag are
 *    fp32 [out].
 *  - dtype selects the storage type of every matrix argument: DORA_BF16 or
 *    DORA_F16.  Arithmetic is fp32 throughout; each stored output is rounded
 *    once, to nearest even.
 *  - All data pointers are DEVICE pointers owned by the caller.  The library
 *    never allocates, frees or synchronises: each call enqueues its kernels on
 *    `stream` and returns.  Scratch memory is passed in by the caller (size from
 *    the *_workspace_bytes queries), so no call makes a transient allocation.
 *  - Return value: DORA_OK, or a status below.  Arguments are validated before
 *    any launch; on a non-zero status nothing was enqueued (except
 *    DORA_HIP_ERROR, reported by the launch itself).  dora_last_error() gives
 *    the message of the calling thread's last failure.
 *  - Any sizes are accepted.  The fast paths need 16-byte aligned pointers and
 *    row lengths that are multiples of 8 elements (for the norm also
 *    in < 2^21); other cases take a slower general path with the same
 *    accuracy (its summation order differs, so results are not bitwise equal
 *    to the fast path's).
 *  - Results are deterministic: no floating-point atomics, fixed reduction
 *    orders, so repeated calls give bitwise identical outputs.
 */
#ifndef DORA_H_
#define DORA_H_

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifndef DORA_API
#define DORA_API __attribute__((visibility("default")))
#endif

#ifdef __cplusplus
extern "C" {
#endif

/*
 * DORA_UNSUPPORTED marks arguments that are valid but that this library does
 * not take; a caller can route such a call elsewhere (the page's eager tier):
 *  - an unknown dtype code;
 *  - sizes whose launch grid would exceed one grid dimension's limit;
 *  - on the fast paths of dora_lora_compose_bwd and dora_norm_bwd, a token or
 *    row slice that would span 2 GiB or more;
 *  - dora_lora_compose_bwd with a shape or pointers its fast path cannot take
 *    and T * r above 2^20 (its slow path runs T * r products in order in one
 *    thread per output column);
 *  - dora_compose_bwd_noalloc with sizes whose partials exceed its scratch;
 *  - in the 8-bit and 4-bit operators (dora_q8_*, dora_q4_*), 2^31 rows or more,
 *    more than 2^22 - 128 columns, or a rank above 2^20;
 *  - in the operators on sorted tokens (dora_adapter_*), more than 2^31 - 1 slots,
 *    1000 adapters or 2^22 columns, or ids of neither 4 nor 8 bytes;
 *  - in both, matrices of so many elements (2^36 and more) that a launch would need
 *    2^32 threads.
 */
enum dora_status {
  DORA_OK = 0,
  DORA_INVALID_ARG = 1, /* null pointer, negative size, workspace too small, bad alias */
  DORA_UNSUPPORTED = 2, /* valid arguments this library does not take (listed above) */
  DORA_HIP_ERROR = 3    /* a kernel launch failed (message from the HIP runtime) */
};

enum dora_dtype { DORA_BF16 = 0, DORA_F16 = 1 };

/*
 * Bytes of device workspace dora_norm_factored needs for these sizes.
 * The scratch is O(out*r + r*r): split-K partial sums of G = A*A^T, the
 * two-term split of (s/2)*G in the storage dtype, and per-split row partials.
 * For every shape it stays within 4*(out*r + r*r) + 64*out bytes, region
 * alignment included (the factored norm's memory bound, paragraph on the
 * factored norm): where the Gram partials would not fit, one K split writes
 * the split of (s/2)*G directly.  Returns 0 for invalid sizes (negative) or an
 * unknown dtype.
 */
DORA_API size_t dora_norm_workspace_bytes(int64_t out, int64_t in, int64_t r, int dtype);

/*
 * norm_out[i] = || W0_i + s * B_i * A ||_2, i in [0, out), in fp32.
 *
 * Computed as sqrt(base_i + cross_i + gram_i) with
 *   base_i  = sum_k W0_ik^2,
 *   cross_i = 2 s * sum_j B_ij * U_ij,   U = W0 * A^T   [out x r],
 *   gram_i  = s^2 * B_i * G * B_i^T,     G = A * A^T    [r x r],
 * (summary page, paragraph on the factored norm).  U and G are dense MFMA
 * contractions with fp32 accumulation; U never leaves the registers.  A
 * negative sum from rounding is clamped to 0.  The norm is a plain value: the
 * backward of the compose treats it as a constant.  With in and r multiples of
 * 8, 16-byte aligned matrices, r <= 32 and out >= 4065 the call is a single
 * launch that forms G itself and leaves ws untouched; the workspace query
 * does not depend on this.
 *
 * W0, A, B: device, dtype.  A and B may be NULL when r == 0.  norm_out: device
 * fp32 [out].  ws: device scratch of at least dora_norm_workspace_bytes(...)
 * bytes, contents undefined on entry and exit; ws may be NULL when that size is
 * 0.  out == 0 is a no-op; in == 0 gives n = 0.
 */
DORA_API int dora_norm_factored(const void* W0, const void* A, const void* B, int64_t out, int64_t in,
                       int64_t r, float s, int dtype, float* norm_out, void* ws, size_t ws_bytes,
                       hipStream_t stream);

/*
 * sq_out[i] = ||W0_i||^2 = sum_k W0_ik^2, i in [0, out), in fp32: the base term
 * of the weight norm on its own.  W0 is frozen during fine-tuning, so this is
 * the cache the summary page proposes as future work (paragraph on
 * limitations: cache the base norm); compute it once and pass it to
 * dora_norm_factored_cached.  One read of W0; squares accumulate in fp32
 * partial sums of at most ceil(in/256) + 1 terms, combined in fp64 and rounded
 * once.
 *
 * W0: device, dtype, [out x in].  sq_out: device fp32 [out], not overlapping
 * W0.  out == 0 is a no-op; in == 0 gives 0.
 */
DORA_API int dora_row_sqnorm(const void* W0, int64_t out, int64_t in, int dtype, float* sq_out,
                             hipStream_t stream);

/*
 * dora_norm_factored with the base term taken from a cache:
 *   norm_out[i] = sqrt(max(base_sq[i] + cross_i + gram_i, 0)),
 * cross_i and gram_i as in dora_norm_factored (summary page, paragraph on
 * limitations: the cached base norm).  With base_sq from dora_row_sqnorm on the
 * same W0 this is ||W0_i + s * B_i * A||_2; the pass over W0 for the cross term
 * then skips the squares.  Same arguments, workspace and errors as
 * dora_norm_factored, plus base_sq: device fp32 [out], not overlapping
 * norm_out or ws (NULL is INVALID_ARG unless out == 0).
 */
DORA_API int dora_norm_factored_cached(const void* W0, const void* A, const void* B, const float* base_sq,
                                       int64_t out, int64_t in, int64_t r, float s, int dtype, float* norm_out,
                                       void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * y = (g - 1) * base + g * s * lora, g_j = mag_j / norm_j broadcast over the T
 * rows (summary page, paragraph on stability near g = 1).  g - 1 is formed as
 * (mag - norm) / norm, whose subtraction is exact when mag/norm is in [1/2, 2],
 * so the base correction is nonzero wherever mag != norm and base != 0.  With
 * add_base != 0, y = base + that delta (the full layer output) in the same
 * pass.  One read of base and lora, one write of y.
 *
 * base, lora, y: device, dtype, [T x out].  mag, norm: device fp32 [out].
 * y may be the same buffer as base or lora (in place); no other overlap.
 * T == 0 or out == 0 is a no-op.  norm_j == 0 follows IEEE division.
 */
DORA_API int dora_compose_fwd(const void* base, const void* lora, const float* mag, const float* norm, float s,
                     int64_t T, int64_t out, int dtype, int add_base, void* y, hipStream_t stream);

/*
 * dora_compose_fwd with the adapter's second projection fused in:
 *   y = (g - 1) * base + g * s * (h * B^T)   (+ base when add_base != 0),
 * where h = x * A^T is the adapter's first projection [T x r] and B is
 * [out x r] (summary page: the fused kernel's gains come from fewer memory
 * accesses).  lora = h * B^T is accumulated in fp32 by MFMA and never stored:
 * one read of base, one write of y, and h and B read per tile (they are small).
 * g - 1 is formed as in dora_compose_fwd; one rounding per output.
 *
 * base, y: device, dtype, [T x out]; h: [T x r]; B: [out x r]; mag, norm:
 * device fp32 [out].  y may be the same buffer as base; no other overlap with
 * an input.  h and B may be NULL when r == 0 (then y is the compose of
 * lora = 0).  T == 0 or out == 0 is a no-op.  The fast path needs out and r
 * multiples of 8, out < 2^22, r <= 2^20 and 16-byte aligned pointers; other
 * cases take a slow path (one thread per output element).
 */
DORA_API int dora_lora_compose_fwd(const void* base, const void* h, const void* B, const float* mag,
                                   const float* norm, float s, int64_t T, int64_t out, int64_t r, int dtype,
                                   int add_base, void* y, hipStream_t stream);

/*
 * Bytes of device workspace dora_norm_bwd needs for these sizes (either
 * path): on the fast path the Gram scratch of the norm, c [out] fp32, the
 * hi/lo pair of s*c*B [out x 2r] and of an r x r product [r x 2r] in the
 * storage dtype, and one fp32 region of row-slice partials of size
 * O(out*r + in*r) reused by the steps in turn.
 * Returns 0 for negative sizes or an unknown dtype.
 */
DORA_API size_t dora_norm_bwd_workspace_bytes(int64_t out, int64_t in, int64_t r, int dtype);

/*
 * Backward of the weight norm n_i = ||W0_i + s * B_i * A||_2 for a caller
 * that does not treat n as a constant (the summary page's paragraph on the
 * factored norm gives its base, cross and Gram parts; the page does not say
 * whether n is differentiated, and dora_compose_bwd takes it as constant).
 * Given dL/dn = d_norm, with c_i = d_norm_i / norm_i (0 where norm_i == 0):
 *   d_B_i = s * c_i * (U_i + s * B_i * G),          U = W0 * A^T, G = A * A^T
 *   d_A   = s * (c .* B)^T * W0 + s^2 * (B^T * diag(c) * B) * A
 * which is s * B^T * dV and s * dV * A^T for dV = c .* (W0 + s * B * A), with
 * the out x in matrix B * A never formed.  W0 is frozen: it gets no gradient.
 * For the DoRA layer, L depends on n only through g = m / n, so
 * d_norm_j = -(m_j / n_j) * d_mag_j with d_mag from dora_compose_bwd.
 * U, G and the two contractions over the out rows run on MFMA with fp32
 * accumulation; the computed operands s*c*B and the r x r product enter them as
 * hi/lo pairs of the storage dtype.  Each output is rounded once.
 *
 * W0: device, dtype, [out x in]; A, d_A: [r x in]; B, d_B: [out x r]; norm
 * (the forward's n) and d_norm: device fp32 [out].  No output overlaps an
 * input, the other output or ws.  ws: at least dora_norm_bwd_workspace_bytes
 * bytes.  r == 0 is a no-op; out == 0 gives d_A = 0; in == 0 gives d_B = 0.
 * The fast path needs in and r multiples of 8, in < 2^21, r <= 2^20 and
 * 16-byte aligned matrix and workspace pointers; other cases take a slow
 * general path (one thread per output element, every sum in order in fp32,
 * no hi/lo operands).
 * In fp16 the fast path stores column j of s*c*B times a power of two
 * sigma_j that puts that column's largest magnitude in [1/2, 1) (sigma_j
 * within 2^-60 .. 2^60; two extra small launches), carries sigma_j on every
 * operand column that feeds row j of d_A, and divides it out of that row in
 * fp32, so a small d_norm, a small B or a single small column of B does not
 * push the operands into fp16's subnormal range.  Entries of the r x r product
 * s*B^T*(c*B) beyond fp16's range (65504) after that scaling still overflow.
 * bf16 has fp32's exponent range and takes sigma_j = 1.
 */
DORA_API int dora_norm_bwd(const void* W0, const void* A, const void* B, const float* norm, const float* d_norm,
                           int64_t out, int64_t in, int64_t r, float s, int dtype, void* d_A, void* d_B, void* ws,
                           size_t ws_bytes, hipStream_t stream);

/*
 * dora_norm_bwd of `out` rows of a W0 that comes in slabs of rows (as an 8-bit
 * one does, unpacked a slab at a time).  d_B holds these rows' gradient; d_A is
 * fp32 [r x in] and, with add_A != 0, is added to (in the order of the calls), so
 * that the sum over all slabs can be rounded once.  The same workspace, sizes and
 * refusals; out == 0 gives d_A = 0 where add_A == 0, else nothing.
 */
DORA_API int dora_norm_bwd_slab(const void* W0, const void* A, const void* B, const float* norm, const float* d_norm,
                                int64_t out, int64_t in, int64_t r, float s, int dtype, int add_A, float* d_A,
                                void* d_B, void* ws, size_t ws_bytes, hipStream_t stream);

/* Bytes of device workspace dora_lora_compose_bwd needs (fp32 slices of dy^T h and column partials). */
DORA_API size_t dora_lora_compose_bwd_workspace_bytes(int64_t T, int64_t out, int64_t r);

/*
 * Backward of dora_lora_compose_fwd for L = sum(dy * y), with norm held
 * constant, never forming lora or d_lora = g * s * dy:
 *   d_base = (g - 1) * dy         (add_base == 0)
 *          = g * dy               (add_base != 0)
 *   d_B    = (g * s * dy)^T h = g * s * (dy^T h)       [out x r]
 *   d_mag_j = (sum_t dy_tj * base_tj + s * sum_k B_jk (dy^T h)_jk) / norm_j,
 * which equals sum_t dy_tj * (base_tj + s * (h B^T)_tj) / norm_j (summary page:
 * the training tier's fused backward; gains from fewer memory accesses).
 * dy^T h is an MFMA contraction over the tokens with fp32 accumulation, its
 * token slices added in a fixed order; d_mag sums its partials in fp64.  The
 * gradient of h, d_lora * B = dy * (g * s * B), is the caller's GEMM.
 *
 * dy, base, d_base: device, dtype, [T x out]; d_base may be NULL (not
 * computed).  h: [T x r]; B, d_B: [out x r].  mag, norm, d_mag: device fp32
 * [out].  No output may overlap an input or another output.  ws: at least
 * dora_lora_compose_bwd_workspace_bytes(T, out, r) bytes on the fast path
 * (out and r multiples of 8, 8 <= r <= 2^20, T >= 1, 16-byte aligned
 * pointers); other cases take a slow path (one thread per output column) and
 * need no workspace; the slow path refuses (DORA_UNSUPPORTED) shapes with
 * T * r > 2^20.  out == 0 is a no-op; T == 0 gives d_B = 0 and d_mag = 0.
 */
DORA_API int dora_lora_compose_bwd(const void* dy, const void* base, const void* h, const void* B, const float* mag,
                                   const float* norm, float s, int64_t T, int64_t out, int64_t r, int dtype,
                                   int add_base, void* d_base, void* d_B, float* d_mag, void* ws, size_t ws_bytes,
                                   hipStream_t stream);

/* Bytes of device workspace dora_compose_bwd needs (per-token-block fp32 partial sums). */
DORA_API size_t dora_compose_bwd_workspace_bytes(int64_t T, int64_t out);

/*
 * Backward of dora_compose_fwd for L = sum(dy * y), with norm held constant:
 *   d_lora = g * s * dy
 *   d_base = (g - 1) * dy         (add_base == 0)
 *          = g * dy               (add_base != 0)
 *   d_mag_j = sum_t dy_tj * (base_tj + s * lora_tj) / norm_j
 * (summary page: fused backward of the training tier; the magnitude gradient is
 * a token reduction whose order may differ from an eager implementation).  The
 * reduction is fixed-order: fp32 partial sums over blocks of tokens, combined
 * in fp64 in a second kernel, so d_mag is bitwise reproducible.
 *
 * dy, base, lora, d_lora, d_base: device, dtype, [T x out]; d_base may be NULL
 * (not computed).  mag, norm, d_mag: device fp32 [out].  d_lora may be the same
 * buffer as dy or lora; d_base may be the same buffer as dy or base; d_lora
 * and d_base must differ.  ws: at least dora_compose_bwd_workspace_bytes(T,
 * out) bytes.  out == 0 is a no-op; T == 0 writes d_mag = 0 / norm.
 */
DORA_API int dora_compose_bwd(const void* dy, const void* base, const void* lora, const float* mag,
                     const float* norm, float s, int64_t T, int64_t out, int dtype, int add_base,
                     void* d_lora, void* d_base, float* d_mag, void* ws, size_t ws_bytes,
                     hipStream_t stream);

/*
 * dora_compose_bwd for callers that cannot allocate device memory (code under
 * stream or graph capture, tight serving loops, harnesses that forbid
 * allocation): same arguments, results and errors, without the workspace.
 * The magnitude-gradient partials go to a scratch array of 24 MiB that the
 * library holds on each GPU it runs on from load until process exit; this
 * call allocates and frees nothing.  Sizes whose partials need more
 * (dora_compose_bwd_workspace_bytes(T, out) > 24 MiB) return DORA_UNSUPPORTED
 * before any launch.  Every call on a GPU shares that GPU's array, so calls
 * that overlap in time on one GPU (on different streams, or from different
 * threads) race on it: serialise them.  The array keeps the last call's
 * partials; each call overwrites every partial it reads.  The first call on a
 * device looks up the array's address there (hipGetSymbolAddress).
 */
DORA_API int dora_compose_bwd_noalloc(const void* dy, const void* base, const void* lora, const float* mag,
                                      const float* norm, float s, int64_t T, int64_t out, int dtype, int add_base,
                                      void* d_lora, void* d_base, float* d_mag, hipStream_t stream);

/*
 * ---- The frozen side in 8 bits -------------------------------------------
 *
 * W0 is frozen and the backward needs x and base only as operands of sums over
 * the tokens, so all three can be held in 8 bits: e4m3 values in blocks of 128
 * with one power-of-two scale 2^e a block.  The entry points below pack and
 * unpack such matrices, multiply with them, and run the compose's backward and
 * the gradient of A from them.
 *
 * Packed rows (activations, gradients), from [rows x cols]:
 *   q  bytes [rows x P], P = cols rounded up to 128, zeros behind cols;
 *   e  bytes [rows x E], E = P / 128 rounded up to 4: byte 127 + e of each block
 *      of 128 columns, 127 behind the last.
 * Packed weight, from [out x in]: blocks of 128 x 128,
 *   q  bytes [out rounded up to 128, x in rounded up to 128], zeros outside;
 *   e  bytes [out / 128 rounded up, x E], as above.
 * e is the smallest exponent >= -126 for which the block's largest finite
 * magnitude is at most 448 * 2^e; the stored value is v * 2^-e rounded once, to
 * nearest even.  A value that is not finite is stored as NaN and does not count
 * for e.  A power of two, because the matrix instruction applies such scales
 * itself, exactly, and because the packed bytes then do not depend on the order
 * of any arithmetic.  q is 16-byte aligned and e 4-byte.  Only bytes written by
 * these entry points (1 to 247) are exponents.
 *
 * Sizes: fewer than 2^31 rows and at most 2^22 - 128 columns (else
 * DORA_UNSUPPORTED).  No output may overlap an input or another output.
 */

/*
 * Pack x [rows x cols] (device, dtype) into q, e.  One read of x, one write of
 * q.  Empty sizes are no-ops.
 */
DORA_API int dora_q8_pack(const void* x, int64_t rows, int64_t cols, int dtype, void* q, void* e, hipStream_t stream);

/* Pack a weight [out x in] into blocks of 128 x 128 (once: the weight is frozen). */
DORA_API int dora_q8_pack_weight(const void* W, int64_t out, int64_t in, int dtype, void* q, void* e,
                                 hipStream_t stream);

/*
 * The values that packed rows (weight == 0) or the first `rows` rows of a
 * packed weight (weight != 0) are held as: x [rows x cols] in dtype.  Exact but
 * for values past the type's range: a block's top rounded up past the largest
 * finite value is held at that value, and bf16 or fp16 subnormals round once.
 */
DORA_API int dora_q8_unpack(const void* q, const void* e, int64_t rows, int64_t cols, int weight, int dtype, void* x,
                            hipStream_t stream);

/* Bytes of device workspace dora_q8_linear_fwd needs (fp32 tiles of a split contraction, often 0). */
DORA_API size_t dora_q8_linear_workspace_bytes(int64_t T, int64_t out, int64_t in);

/*
 * y [T x out] = x W0^T from packed rows x [T x in] and a packed weight
 * [out x in]: y_tj = sum over the blocks of 2^(e_x + e_W) * (sum of the block's
 * products), rounded once to dtype.  The sums are fp32, but not every product
 * enters them whole: the 8-bit matrix instruction cuts the eight products of
 * eight consecutive k, towards zero, to multiples of 2^-13 times the power of two
 * of the largest one's operand exponents before it adds them.  So
 *   |y - exact| <= half a step of dtype + in * 2^-23 * sum |x_k W_k|
 *                + 7 * 2^-13 * sum over the eights of max |x_k| * max |W_k|;
 * measured, the cut is 1.5e-5 to 6.5e-5 of the norm of y, and adds 2 % to the
 * error of an fp16 result against 64 bits, 0.04 % to a bf16 one's.  A caller who
 * needs fp32 products unpacks the operands (exact in bf16) and multiplies those.
 * The frozen layer's base product of the training and the inference tier; for few rows (T <= 64, as when single
 * tokens are generated) the weight is streamed once and the rows share it.
 * in == 0 gives y = 0.  A NaN in a row of x gives NaN in that row of y alone.
 * ws: 16-byte aligned, at least dora_q8_linear_workspace_bytes bytes.
 */
DORA_API int dora_q8_linear_fwd(const void* xq, const void* xe, const void* wq, const void* we, int64_t T, int64_t out,
                                int64_t in, int dtype, void* y, void* ws, size_t ws_bytes, hipStream_t stream);

/* Bytes of device workspace dora_q8_linear_bwd needs. */
DORA_API size_t dora_q8_linear_bwd_workspace_bytes(int64_t T, int64_t out, int64_t in);

/*
 * dx [T x in] = g W0 from packed rows g [T x out] and the same packed weight
 * (its transpose is not stored: the kernel's reads transpose it), with the sums
 * and the bound of dora_q8_linear_fwd, the eights along out.  W0 is frozen, so
 * there is no gradient of the weight.  out == 0 gives dx = 0.
 */
DORA_API int dora_q8_linear_bwd(const void* gq, const void* ge, const void* wq, const void* we, int64_t T, int64_t out,
                                int64_t in, int dtype, void* dx, void* ws, size_t ws_bytes, hipStream_t stream);

/* Bytes of device workspace dora_q8_lora_compose_bwd needs (fp32 slices, column partials, padded copies). */
DORA_API size_t dora_q8_lora_compose_bwd_workspace_bytes(int64_t T, int64_t out, int64_t r);

/*
 * dora_lora_compose_bwd with the base from packed rows [T x out] (the forward's
 * base, kept in 8 bits until the backward): the same formulas for d_base, d_B
 * and d_mag, base being the values the rows are held as.  d_base is written in
 * dtype to d_base, or packed straight from fp32 to (dq, de) as dora_q8_pack
 * would of the unrounded product, which is what dora_q8_linear_bwd takes; either
 * or both may be NULL (dq and de together).
 *
 * dy [T x out], h [T x r], B, d_B [out x r], d_base: device, dtype, 16-byte
 * aligned; any sizes (rows that are not multiples of 8 elements are copied into
 * the workspace first).  r == 0 is lora = 0.  out == 0 is a no-op; T == 0 gives
 * d_B = 0 and d_mag = 0 / norm.  r <= 2^20, else DORA_UNSUPPORTED.
 */
DORA_API int dora_q8_lora_compose_bwd(const void* dy, const void* bq, const void* be, const void* h, const void* B,
                                      const float* mag, const float* norm, float s, int64_t T, int64_t out, int64_t r,
                                      int dtype, int add_base, void* d_base, void* dq, void* de, void* d_B,
                                      float* d_mag, void* ws, size_t ws_bytes, hipStream_t stream);

/* Bytes of device workspace dora_q8_grad_a needs (fp32 slices of x^T d_h, a padded copy of d_h). */
DORA_API size_t dora_q8_grad_a_workspace_bytes(int64_t T, int64_t in, int64_t r);

/*
 * d_A [r x in] = d_h^T x, the gradient of the adapter's first projection h = x
 * A^T, from x kept in packed rows [T x in] since the forward.  x enters the
 * products as dora_q8_unpack gives it in dtype, d_h [T x r] (device, dtype,
 * 16-byte aligned) as it is; fp32 sums, token slices added in a fixed order,
 * rounded once.  in == 0 or r == 0 is a no-op; T == 0 gives d_A = 0.  r <= 2^20,
 * else DORA_UNSUPPORTED.
 */
DORA_API int dora_q8_grad_a(const void* dh, const void* xq, const void* xe, int64_t T, int64_t in, int64_t r, int dtype,
                            void* d_A, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * ---- The frozen weight in 4 bits ------------------------------------------
 *
 * W0 [out x in] in blocks of 32 consecutive columns of a row: e2m1 values (0, 0.5,
 * 1, 1.5, 2, 3, 4, 6 and their negatives) with one power-of-two scale 2^e a block,
 * the smallest e in [-23, 13] for which the block's largest magnitude is at most
 * 7 * 2^e.  The value held is v * 2^-e rounded to the nearest e2m1 value, ties to
 * the one of even code, 6 at most, times 2^e: exact in bf16 and in fp16.
 * Magnitudes below 2^-25 are held as 0, and 6 * 2^13 is the largest.  A block with
 * a value that is not finite is NaN as a whole.  17 bits hold 4 values.
 *
 * Layout: tiles of 32 rows x 64 columns, zeros outside W0, row tiles outermost,
 *   q  bytes [out / 32 rounded up, in / 64 rounded up, 1024],
 *   e  bytes [out / 32 rounded up, in / 64 rounded up, 64].
 * Row 8g + i (g < 4, i < 8) of a tile has its block b (of two) in the 16 bytes of q
 * at 128 i + 32 g + 16 (b ^ (i/2 % 2)), codes of 4 bits (sign above the magnitude's
 * number in the list above), even columns in the low halves, and the byte 127 + e
 * (255: NaN) in e at 32 b + 8 g + 2 (i % 4) + i/4.  q and e are 16-byte aligned.
 * Only bytes written by dora_q4_pack_weight are valid ones.
 *
 * Sizes: fewer than 2^31 rows of x, at most 2^22 - 128 rows and columns of W0 and
 * 2^31 - 1 tiles (else DORA_UNSUPPORTED).  No output may overlap an input or
 * another output.
 */

/* Pack W [out x in] (device, dtype) into q, e (once: it is frozen).  Empty sizes are no-ops. */
DORA_API int dora_q4_pack_weight(const void* W, int64_t out, int64_t in, int dtype, void* q, void* e,
                                 hipStream_t stream);

/* The values that the first `rows` rows of a packed weight of `cols` columns are held as, in dtype (exact). */
DORA_API int dora_q4_unpack_weight(const void* q, const void* e, int64_t rows, int64_t cols, int dtype, void* W,
                                   hipStream_t stream);

/* Bytes of device workspace dora_q4_linear_fwd needs (fp32 tiles of a split contraction, rows padded to 8; often 0). */
DORA_API size_t dora_q4_linear_workspace_bytes(int64_t T, int64_t out, int64_t in);

/*
 * y [T x out] = x W0^T with x [T x in] (device, dtype, 16-byte aligned) and a packed
 * weight: 16-bit operands, products and sums in fp32, rounded once to dtype.  For
 * few rows (single tokens as they are generated) the weight is streamed once.
 * in == 0 gives y = 0.  A NaN in a row of x gives NaN in that row of y alone, a NaN
 * block of W0 in its column of y.  ws: 16-byte aligned, at least
 * dora_q4_linear_workspace_bytes bytes.
 */
DORA_API int dora_q4_linear_fwd(const void* x, const void* q, const void* e, int64_t T, int64_t out, int64_t in,
                                int dtype, void* y, void* ws, size_t ws_bytes, hipStream_t stream);

/* Bytes of device workspace dora_q4_linear_bwd needs. */
DORA_API size_t dora_q4_linear_bwd_workspace_bytes(int64_t T, int64_t out, int64_t in);

/*
 * dx [T x in] = g W0 with g [T x out] and the same packed weight, which is
 * transposed on the way to the matrix instructions.  W0 is frozen, so there is no
 * gradient of the weight.  out == 0 gives dx = 0.
 */
DORA_API int dora_q4_linear_bwd(const void* g, const void* q, const void* e, int64_t T, int64_t out, int64_t in,
                                int dtype, void* dx, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * The kernel that a call's sizes ask for, on the host: tests name with it what they
 * run, and sweeps what they time.  product 0: dora_q4_linear_fwd of T rows, 1:
 * dora_q4_linear_bwd, 2: the product in dora_q4_norm_cached (T: the rank).  plan [6]:
 *   0  rows of a tile; 0 for the kernels for few rows
 *   1  columns of a tile; for few rows, of a workgroup's group
 *   2  tiles that fill whole rounds of workgroups, each with its whole contraction
 *   3  the other tiles (for few rows: all groups)
 *   4  ranges of the contraction of these
 *   5  workgroups
 * All zeros for an empty product, which a fill kernel takes.  The choice is no part of
 * the interface: another version may take others.
 */
DORA_API int dora_q4_plan(int64_t T, int64_t out, int64_t in, int product, int64_t* plan);

/* Bytes of device workspace dora_q4_norm_cached needs (0 for sizes that it does not take). */
DORA_API size_t dora_q4_norm_workspace_bytes(int64_t out, int64_t in, int64_t r, int dtype);

/*
 * dora_norm_factored_cached of a packed weight: norm_out [out] (fp32) = ||W0 + s * B * A||
 * per row, with ||W0_i||^2 of the values held from base_sq (fp32).  W0 is not unpacked:
 * the product W0 A^T keeps its fp32 sums in the workspace.  A [r x in], B [out x r] and
 * ws are 16-byte aligned, in and r multiples of 8, in below 2^21 and 0 < r <= 512 (else
 * DORA_UNSUPPORTED: unpack rows and use dora_norm_factored_cached).  No output may
 * overlap an input or another output.
 */
DORA_API int dora_q4_norm_cached(const void* q, const void* e, const void* A, const void* B, const float* base_sq,
                                 int64_t out, int64_t in, int64_t r, float s, int dtype, float* norm_out, void* ws,
                                 size_t ws_bytes, hipStream_t stream);

/*
 * ---- Tokens sorted by adapter ---------------------------------------------
 *
 * Several adapters over one W0: token t of a batch has k slots (t, j), each with
 * the number of an adapter in [0, n), or any other number for none.  Slots are
 * numbered t * k + j.  Each slot owns one of R = T k rows: rows are sorted by
 * adapter, an adapter's rows in the order of its slots, and the rows of slots
 * without one come last.
 *   order [R]      the slot of each row; the complement ~slot (negative) where the
 *                  slot has no adapter;
 *   place [T x k]  the row of each slot; its complement where it has none;
 *   bounds [n + 1] adapter a has rows [bounds[a], bounds[a + 1]).
 * The operators on rows take place as dora_adapter_sort leaves it.  (Numbers
 * outside [-R, R) in it are left out, so that no call reads or writes beyond its
 * matrices; a row that no slot owns is then not written.)
 *
 * Sizes: at most 2^31 - 1 slots, 1000 adapters, rows of 2^22 elements (else
 * DORA_UNSUPPORTED).  Matrices are device, dtype, row-major; any alignment of their
 * elements is taken, 16 bytes and D % 8 == 0 faster.  No output may overlap an
 * input or another output, but y of dora_adapter_combine may be base itself.
 */

/* Bytes of device workspace dora_adapter_sort needs (counts of its workgroups; 0 for up to 4096 slots). */
DORA_API size_t dora_adapter_sort_workspace_bytes(int64_t T, int64_t k, int64_t n);

/* ids [T x k]: device, int64 (id_bytes 8) or int32 (4).  order, place, bounds: device int32.  No slots: bounds = 0. */
DORA_API int dora_adapter_sort(const void* ids, int id_bytes, int64_t T, int64_t k, int64_t n, int32_t* order,
                               int32_t* place, int32_t* bounds, void* ws, size_t ws_bytes, hipStream_t stream);

/* rows [T k x D]: the row of slot (t, j) is x[t], zeros for a slot without an adapter. */
DORA_API int dora_adapter_gather(const void* x, const int32_t* place, int64_t T, int64_t k, int64_t D, int dtype,
                                 void* rows, hipStream_t stream);

/*
 * y[t] = base[t] + sum over the slots j with an adapter of weights[t, j] * (their
 * rows), in fp32, rounded once.  weights: fp32 [T x k], NULL for ones; base: NULL
 * for zeros.  What stands in the rows and weights of other slots is not used.
 * Without weights and base this is the gradient of dora_adapter_gather.
 */
DORA_API int dora_adapter_combine(const void* rows, const float* weights, const int32_t* place, const void* base,
                                  int64_t T, int64_t k, int64_t D, int dtype, void* y, hipStream_t stream);

/*
 * The gradients of dora_adapter_combine: d_rows [T k x D], the row of slot (t, j)
 * weights[t, j] * dy[t], and d_weights [T x k] (fp32) = <dy[t], that row of rows>;
 * both zeros for a slot without an adapter.  Either may be NULL (not computed), and
 * rows without d_weights.  The gradient of base is dy.
 */
DORA_API int dora_adapter_combine_bwd(const void* dy, const void* rows, const float* weights, const int32_t* place,
                                      int64_t T, int64_t k, int64_t D, int dtype, void* d_rows, float* d_weights,
                                      hipStream_t stream);

/* Message of the calling thread's last non-OK status ("" if none).  Valid until the next call. */
DORA_API const char* dora_last_error(void);

/* Library build string (version, target architecture). */
DORA_API const char* dora_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DORA_H_ */
