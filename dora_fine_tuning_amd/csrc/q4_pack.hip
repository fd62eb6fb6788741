// Packing of a 16-bit weight into 4-bit blocks, and back, for gfx950.
//
// One pass each, bound by HBM: packing reads 2 bytes and writes 17/32 an element,
// unpacking the reverse.  A block of 32 is 4 lanes of 8 values (one 16-byte load
// each); a workgroup's 256 lanes are one tile of 32 x 64, and take kU tiles of a
// row of tiles, all loads in flight before the first maximum.
//
// 27648 x 5120 in bf16 (358 MB): packing 66 us (5.4 TB/s), unpacking 53 to 68; 8192^2
// (170 MB): 26.6 and 27.2 (6.3 TB/s), where a copy of 2 GiB reaches 4.9.
#include "q4_common.hpp"

namespace dora {

namespace {

constexpr int kU = 4;

// Lane coordinates within a tile: row 8g + i, eight columns from 8 * c on.
struct At {
  uint32_t c, g, i;
};
__device__ inline At lane_at() { return At{threadIdx.x & 7, (threadIdx.x >> 3) & 3, threadIdx.x >> 5}; }
__device__ inline uint32_t q_byte(const At& a) { return q4_unit(a.i, a.g, a.c >> 2) + 4 * (a.c & 3); }
__device__ inline uint32_t e_byte(const At& a) { return 32 * (a.c >> 2) + 8 * a.g + 2 * (a.i & 3) + (a.i >> 2); }

template <int DT, bool VEC>
__global__ __launch_bounds__(256) void q4_pack_k(const void* W, int64_t out, int64_t in, uint32_t ib, uint32_t groups,
                                                 uint8_t* q, uint8_t* e) {
  using T16 = typename Dt<DT>::T;
  const At a = lane_at();
  const uint32_t rt = blockIdx.x / groups, t0 = (blockIdx.x - rt * groups) * kU;
  const int64_t row = static_cast<int64_t>(rt) * kQ4Rows + 8 * a.g + a.i;
  const T16* src = static_cast<const T16*>(W) + row * in;
  Chunk c[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t col = static_cast<int64_t>(t0 + u) * kQ4Cols + 8 * a.c;
    if constexpr (VEC) {  // in % 8 == 0: a chunk is inside or outside as a whole
      c[u] = row < out && col < in ? *reinterpret_cast<const Chunk*>(src + col) : zero_chunk();
    } else {
      typename Dt<DT>::V8 v;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = row < out && col + j < in ? src[col + j] : static_cast<T16>(0.0f);
      c[u] = __builtin_bit_cast(Chunk, v);
    }
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    if (t0 + u >= ib) break;
    float v[8];
    chunk_to_f32<DT>(c[u], v);
    // the bits of magnitudes order as they do, infinity and then NaN above all
    int m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __builtin_bit_cast(int, v[j]) & 0x7fffffff);
    m = max(m, __builtin_amdgcn_update_dpp(0, m, 0xb1, 0xf, 0xf, false));  // quad_perm 1 0 3 2
    m = max(m, __builtin_amdgcn_update_dpp(0, m, 0x4e, 0xf, 0xf, false));  // quad_perm 2 3 0 1
    const bool bad = m >= 0x7f800000;
    const uint32_t byte = bad ? 255u : q4_exp_byte(static_cast<uint32_t>(m));
    const uint32_t w = bad ? 0u : q4_encode8(v, q4_scale(byte));
    const int64_t tile = static_cast<int64_t>(rt) * ib + t0 + u;
    *reinterpret_cast<uint32_t*>(q + tile * kQ4TileQ + q_byte(a)) = w;
    if ((a.c & 3) == 0) e[tile * kQ4TileE + e_byte(a)] = static_cast<uint8_t>(byte);
  }
}

template <int DT, bool VEC>
__global__ __launch_bounds__(256) void q4_unpack_k(const uint8_t* q, const uint8_t* e, int64_t rows, int64_t cols,
                                                   uint32_t ib, uint32_t groups, void* x) {
  using T16 = typename Dt<DT>::T;
  const At a = lane_at();
  const uint32_t rt = blockIdx.x / groups, t0 = (blockIdx.x - rt * groups) * kU;
  const int64_t row = static_cast<int64_t>(rt) * kQ4Rows + 8 * a.g + a.i;
  uint32_t w[kU], b[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t tile = static_cast<int64_t>(rt) * ib + min(t0 + u, ib - 1);
    w[u] = *reinterpret_cast<const uint32_t*>(q + tile * kQ4TileQ + q_byte(a));
    b[u] = e[tile * kQ4TileE + e_byte(a)];
  }
  if (row >= rows) return;
  T16* dst = static_cast<T16*>(x) + row * cols;
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t col = static_cast<int64_t>(t0 + u) * kQ4Cols + 8 * a.c;
    const Chunk c = q4_decode8<DT>(w[u], q4_scale(b[u]));
    if constexpr (VEC) {
      if (col < cols) *reinterpret_cast<Chunk*>(dst + col) = c;
    } else {
      const auto v = __builtin_bit_cast(typename Dt<DT>::V8, c);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col + j < cols) dst[col + j] = v[j];
    }
  }
}

}  // namespace

int64_t q4_pack_grid(int64_t out, int64_t in) {
  return q4_ceil(out, kQ4Rows) * q4_ceil(q4_ceil(in, kQ4Cols), kU);
}

hipError_t launch_q4_pack(const void* W, int64_t out, int64_t in, int dtype, bool vec, void* q, void* e,
                          hipStream_t stream) {
  const uint32_t ib = static_cast<uint32_t>(q4_ceil(in, kQ4Cols)), groups = (ib + kU - 1) / kU;
  const dim3 grid(static_cast<uint32_t>(q4_pack_grid(out, in)));
  auto go = [&](auto k) {
    hipLaunchKernelGGL(k, grid, dim3(256), 0, stream, W, out, in, ib, groups, static_cast<uint8_t*>(q),
                       static_cast<uint8_t*>(e));
  };
  if (dtype == 0)
    vec ? go(q4_pack_k<0, true>) : go(q4_pack_k<0, false>);
  else
    vec ? go(q4_pack_k<1, true>) : go(q4_pack_k<1, false>);
  return hipGetLastError();
}

hipError_t launch_q4_unpack(const void* q, const void* e, int64_t rows, int64_t cols, int dtype, bool vec, void* x,
                            hipStream_t stream) {
  const uint32_t ib = static_cast<uint32_t>(q4_ceil(cols, kQ4Cols)), groups = (ib + kU - 1) / kU;
  const dim3 grid(static_cast<uint32_t>(q4_pack_grid(rows, cols)));
  auto go = [&](auto k) {
    hipLaunchKernelGGL(k, grid, dim3(256), 0, stream, static_cast<const uint8_t*>(q), static_cast<const uint8_t*>(e),
                       rows, cols, ib, groups, x);
  };
  if (dtype == 0)
    vec ? go(q4_unpack_k<0, true>) : go(q4_unpack_k<0, false>);
  else
    vec ? go(q4_unpack_k<1, true>) : go(q4_unpack_k<1, false>);
  return hipGetLastError();
}

}  // namespace dora
