// The 8-bit block format and what its kernels share.
//
// Values are OCP e4m3 with a power-of-two scale 2^e for each block of 128: a
// block is 128 consecutive columns of one row (activations, gradients), or a
// 128 x 128 tile (the frozen weight).  Rows are padded with zeros to whole
// blocks, a weight also to whole tiles of rows.  Exponents are bytes 127 + e,
// one row of them per row of blocks, padded to a multiple of four bytes.
//
// Why a power of two: the scaled matrix instruction of gfx950 takes exactly
// such bytes and applies them itself, so a product needs no scaling between
// blocks; the scaling is exact in every type involved, so the stored bits do
// not depend on the order of any arithmetic; and e4m3 is a floating-point type,
// so a finer scale would buy at most part of one binade at a block's bottom.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dora_common.hpp"

namespace dora {

constexpr int64_t kQ8Block = 128;

__host__ __device__ inline int64_t q8_ceil(int64_t n, int64_t k) { return (n + k - 1) / k; }
// bytes of a packed row of n columns, and of its exponent row
__host__ __device__ inline int64_t q8_row_bytes(int64_t n) { return q8_ceil(n, kQ8Block) * kQ8Block; }
__host__ __device__ inline int64_t q8_exp_bytes(int64_t n) { return q8_ceil(q8_ceil(n, kQ8Block), 4) * 4; }

// The exponent byte 127 + e of a block whose largest finite magnitude is amax:
// the smallest e >= -126 with amax * 2^-e <= 448 = 1.75 * 2^8.
__device__ inline uint32_t q8_exp_byte(float amax) {
  const uint32_t u = __builtin_bit_cast(uint32_t, amax);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>((e < -126 ? -126 : e) + 127);
}
// 2^e for a byte in [1, 247]
__device__ inline float q8_scale(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }

// Eight values times 2^-e, rounded to nearest even e4m3 (values that are not
// finite give NaN); |v| * 2^-e is at most 448 where it is finite.  The conversion
// divides by its scale operand, a power of two, exactly.
__device__ inline uint2 q8_encode8(const float (&v)[8], float scale) {
  typedef short s2 __attribute__((ext_vector_type(2)));
  s2 lo = {0, 0}, hi = {0, 0};
  lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, v[0], v[1], scale, false);
  lo = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(lo, v[2], v[3], scale, true);
  hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, v[4], v[5], scale, false);
  hi = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(hi, v[6], v[7], scale, true);
  return uint2{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
}

typedef float q8_f2 __attribute__((ext_vector_type(2)));
// Eight e4m3 values times 2^e, in fp32.
__device__ inline void q8_decode8(uint2 q, float scale, float (&f)[8]) {
  const q8_f2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q.x, scale, false);
  const q8_f2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q.x, scale, true);
  const q8_f2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q.y, scale, false);
  const q8_f2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q.y, scale, true);
  f[0] = a[0], f[1] = a[1], f[2] = b[0], f[3] = b[1], f[4] = c[0], f[5] = c[1], f[6] = d[0], f[7] = d[1];
}

// A value past the type's largest (a block's top rounded up) is held at it; NaN stays.
template <int DT>
__device__ inline float q8_hold1(float f) {
  constexpr float big = DT == 0 ? 3.3895313892515355e38f : 65504.0f;
  f = f > big ? big : f;
  return f < -big ? -big : f;
}
template <int DT>
__device__ inline void q8_hold(float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = q8_hold1<DT>(f[i]);
}

// A maximum leaves out a quiet NaN, but gives a signaling one, quieted, in place
// of the other operands, and the next maximum then drops it with all that was
// gathered before.  Arithmetic results and values converted from fp16 are quiet;
// bf16 reaches fp32 by a shift, with the bits that memory holds.  (Packing 10240 x
// 27648 takes 149 us with and without; 8192^2 out of the caches 31.5 and 30.8.)
template <int DT>
__device__ inline void q8_quiet(float (&v)[8]) {
  if constexpr (DT == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __builtin_canonicalizef(v[i]);
  }
}
// max(m, |a|, |b|), quiet NaN left out
__device__ inline float q8_max3(float m, float a, float b) {
  float r;
  asm("v_max3_f32 %0, %1, abs(%2), abs(%3)" : "=v"(r) : "v"(m), "v"(a), "v"(b));
  return r;
}
// Largest magnitude among eight values (no signaling NaN), NaN left out; infinite if one is.
__device__ inline float q8_amax8(const float (&v)[8]) {
  return q8_max3(q8_max3(q8_max3(q8_max3(0.0f, v[0], v[1]), v[2], v[3]), v[4], v[5]), v[6], v[7]);
}
// Maximum over each group of 16 lanes, of numbers >= 0 (whose bits order as they do).
__device__ inline float q8_max16(float a) {
  int x = __builtin_bit_cast(int, a);
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x128, 0xf, 0xf, false));  // row_ror:8
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x124, 0xf, 0xf, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x122, 0xf, 0xf, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x121, 0xf, 0xf, false));
  return __builtin_bit_cast(float, x);
}
// Largest finite magnitude among the eight values of each of 16 lanes.
__device__ inline float q8_block_amax(const float (&v)[8]) {
  const float inf = __builtin_inff();
  float a = q8_max16(q8_amax8(v));
  if (__any(a == inf)) {  // rare: once more without the infinite ones
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = __builtin_fabsf(v[i]);
      m = x < inf && x > m ? x : m;
    }
    a = q8_max16(m);
  }
  return a;
}

// ---- host-side launch interface

hipError_t launch_q8_pack(const void* x, int64_t rows, int64_t cols, int dtype, bool vec, void* q, void* e,
                          hipStream_t stream);
hipError_t launch_q8_pack_tiles(const void* W, int64_t out, int64_t in, int dtype, bool vec, void* q, void* e,
                                hipStream_t stream);
hipError_t launch_q8_unpack(const void* q, const void* e, int64_t rows, int64_t cols, bool tiles, int dtype, bool vec,
                            void* x, hipStream_t stream);

// Products with the packed weight.  trans = false: y [T x out] = x W^T
// (contraction over in); trans = true: dx [T x in] = g W (over out).
struct Q8GemmArgs {
  const void *xq, *xe, *wq, *we;
  int64_t T, out, in;
  int dtype;
  bool trans;
  void* y;
  void* ws;
  hipStream_t stream;
};
size_t q8_gemm_workspace_bytes(int64_t T, int64_t out, int64_t in, bool trans);
int64_t q8_gemm_max_grid(int64_t T, int64_t out, int64_t in, bool trans);
hipError_t launch_q8_gemm(const Q8GemmArgs& a);

// Backward from 8-bit blocks: the compose's (base packed) and A's (x packed).
struct Q8ComposeBwdArgs {
  const void *dy, *bq, *be, *h, *B;
  const float *mag, *norm;
  float s;
  int64_t T, out, r;
  int dtype, add_base;
  void *d_base, *dq, *de;  // d_base in 16 bits, or packed (either or both may be null)
  void* d_B;
  float* d_mag;
  void* ws;
  hipStream_t stream;
};
struct Q8GradAArgs {
  const void *dh, *xq, *xe;
  int64_t T, in, r;
  int dtype;
  void* d_A;
  void* ws;
  hipStream_t stream;
};
struct Q8BwdSizes {
  size_t bytes = 0;  // of the workspace
  int64_t grid = 0;  // largest grid dimension, or a bound of it
};
// nx: columns contracted against (out of the compose's backward, in of A's).
Q8BwdSizes q8_bwd_sizes(int64_t T, int64_t nx, int64_t r, bool compose);
hipError_t launch_q8_compose_bwd(const Q8ComposeBwdArgs& a);
hipError_t launch_q8_grad_a(const Q8GradAArgs& a);

}  // namespace dora
