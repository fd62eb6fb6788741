// The 4-bit block format of the frozen weight and what its kernels share.
//
// A block is 32 consecutive columns of one row: OCP e2m1 values (0, 0.5, 1, 1.5,
// 2, 3, 4, 6 and their negatives) with one power-of-two scale 2^e, e in [-23, 13].
// e is the smallest for which the block's largest magnitude is at most 7 * 2^e:
// up to 7 the nearest of the type's values is its largest, 6, and no further off
// than half a step.  The range of e is that for which every value, 0.5 * 2^-23 to
// 6 * 2^13, is exact in fp16 (its subnormals included) and in bf16, so that one
// packed weight serves both and the products' operands carry no second rounding.
//
// Why this type: the conversion instructions of gfx950 take a byte of two such
// values and a power of two and give two bf16 or fp16 values, so that a weight
// costs half an instruction a value on its way from 4 bits to a matrix operand.
// Root mean square error on normal values: 11.2 % of theirs (11.5 % with a limit
// of 6 instead of 7; a 4-bit integer with a 16-bit scale per 64 values, as many
// bits, 10.8 %).
//
// Layout: tiles of 32 rows x 64 columns, zeros outside the weight, row tiles
// outermost.  A tile's q are 1024 bytes, its exponent bytes 127 + e (255: a block
// with a value that is not finite, NaN as a whole) 64.  Row 8g + i (g < 4, i < 8)
// keeps its block b (of two) in the 16 bytes at 128 i + 32 g + 16 (b ^ (i/2 % 2)),
// even columns in the low halves, and its exponent at 32 b + 8 g + 2 (i % 4) + i/4.
// So a stage of a product (64 columns of 32 rows, or 32 rows of 64 columns) is one
// piece of memory that goes to LDS as it is; there, the 16 lanes that read 16
// different rows of a block (the forward) or one row of each eight (the backward)
// meet 16 different bank groups; and the rows 8g .. 8g + 7 that one lane of a
// matrix result holds leave as one 16-byte store.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dora_common.hpp"

namespace dora {

constexpr int64_t kQ4Rows = 32, kQ4Cols = 64;  // a tile
constexpr int64_t kQ4TileQ = 1024, kQ4TileE = 64;

__host__ __device__ inline int64_t q4_ceil(int64_t n, int64_t k) { return (n + k - 1) / k; }

// Byte of a tile where row 8g + i has its block b; rows i and i + 4 are 512 apart.
__device__ inline uint32_t q4_unit(uint32_t i, uint32_t g, uint32_t b) {
  return 128 * i + 32 * g + 16 * (b ^ ((i >> 1) & 1));
}

// The exponent byte of a block whose largest magnitude has these (finite) bits.
__device__ inline uint32_t q4_exp_byte(uint32_t bits) {
  const int e = static_cast<int>(bits >> 23) - 127 - 2 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);  // 7 = 1.75 * 2^2
  return static_cast<uint32_t>((e < -23 ? -23 : e > 13 ? 13 : e) + 127);
}
// 2^e for a byte in [104, 140]; infinite for 255, which the conversions take as NaN.
__device__ inline float q4_scale(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }

// Eight values times 2^-e as e2m1, nearest, ties to even, 6 at most.
__device__ inline uint32_t q4_encode8(const float (&v)[8], float scale) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
  return w;
}

// The two values in byte B of w times 2^e, as a pair of the storage type (exact).
template <int DT, int B>
__device__ inline uint32_t q4_decode2(uint32_t w, float scale) {
  if constexpr (DT == 0)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, B));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, scale, B));
}
template <int DT>
__device__ inline Chunk q4_decode8(uint32_t w, float scale) {
  Chunk c;
  c.w[0] = q4_decode2<DT, 0>(w, scale);
  c.w[1] = q4_decode2<DT, 1>(w, scale);
  c.w[2] = q4_decode2<DT, 2>(w, scale);
  c.w[3] = q4_decode2<DT, 3>(w, scale);
  return c;
}

// ---- host-side launch interface

int64_t q4_pack_grid(int64_t out, int64_t in);  // workgroups of 256, of either
hipError_t launch_q4_pack(const void* W, int64_t out, int64_t in, int dtype, bool vec, void* q, void* e,
                          hipStream_t stream);
hipError_t launch_q4_unpack(const void* q, const void* e, int64_t rows, int64_t cols, int dtype, bool vec, void* x,
                            hipStream_t stream);

// Products with the packed weight.  trans = false: y [T x out] = x W^T
// (contraction over in); trans = true: dx [T x in] = g W (over out).
struct Q4GemmArgs {
  const void *x, *wq, *we;
  int64_t T, out, in;
  int dtype;
  bool trans;
  void* y;
  void* ws;
  hipStream_t stream;
};
// The kernel a call takes and how it shares out its work.
struct Q4Plan {
  enum Path { kLow, kThin, kFlat, kBroad, kWide, kFew } path = kWide;
  int64_t N = 0, K = 0, xp = 0;  // output columns, contraction, elements of a row of x in the workspace or as given
  int R = 1;                     // row tiles of a group of few rows
  int S = 0, nSplit = 1;         // stages of 64; ranges of them
  int64_t nRB = 0, nTiles = 0, whole = 0, grid = 0;
  size_t pad = 0, bytes = 0;  // of padded rows; of a split's fp32 sums
  bool parts = false;         // the sums stay in the workspace, for q4_norm.hip
  size_t workspace() const { return pad + bytes; }
  // units of work (tiles in up to 16 ranges) are numbered in 32 bits
  int64_t units() const { return nRB * nTiles * 16 > grid ? nRB * nTiles * 16 : grid; }
};
Q4Plan q4_plan(int64_t T, int64_t out, int64_t in, bool trans);
hipError_t launch_q4_gemm(const Q4GemmArgs& a, const Q4Plan& plan);
void q4_plan_numbers(const Q4Plan& p, bool trans, int64_t* n);  // as dora_q4_plan gives them

// Where a forward product leaves its sums if they stay in the workspace: entries of 64
// register quads, one of each lane, for 16 rows of x and, with half h, the output columns
// 32 rt + 8 (lane / 16) + 4 h + register.
struct Q4Parts {
  int few, nSplit;
  int64_t all;  // groups or tiles of a range
  int R, NT;                                  // few rows: row and token tiles of a group
  int WM, WN, TMW, TNW, nRB, nTiles, group;   // tiles
};
Q4Plan q4_parts_plan(Q4Plan p, int64_t T);  // from q4_plan's
Q4Parts q4_parts_of(const Q4Plan& p, int64_t T);

// The norm of a packed weight with an adapter (q4_norm.hip).  ghi, glo: (s/2) A A^T.
struct Q4NormArgs {
  const void *B, *ghi, *glo;
  const float *base_sq, *part;
  int64_t out, r;
  int dtype;
  float s;
  float* norm;
  hipStream_t stream;
};
hipError_t launch_q4_norm_join(const Q4NormArgs& a, const Q4Parts& parts);

}  // namespace dora
