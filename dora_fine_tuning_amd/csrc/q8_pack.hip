// Packing of 16-bit matrices into 8-bit blocks, and back, for gfx950.
//
// One pass each, bound by HBM: packing reads 2 bytes and writes 1 + 1/128 an
// element, unpacking the reverse.  A block of 128 is 16 lanes of 8 values (one
// 16-byte load each): its largest magnitude is four lane exchanges away, and
// its values never leave the registers between the maximum and the rounding.
#include <type_traits>

#include "q8_common.hpp"

namespace dora {

namespace {

// Blocks a 16-lane group takes, all loads in flight before the first maximum.
constexpr int kU = 4;

template <int DT, bool VEC>
__device__ inline Chunk load8(const void* x, int64_t row, int64_t col, int64_t cols) {
  using T16 = typename Dt<DT>::T;
  const T16* p = static_cast<const T16*>(x) + row * cols + col;
  if constexpr (VEC) {  // cols % 8 == 0: a chunk is inside or outside as a whole
    return col < cols ? *reinterpret_cast<const Chunk*>(p) : zero_chunk();
  } else {
    typename Dt<DT>::V8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = col + i < cols ? p[i] : static_cast<T16>(0.0f);
    return __builtin_bit_cast(Chunk, v);
  }
}

template <int DT, bool VEC>
__global__ __launch_bounds__(256) void q8_pack_rows(const void* x, uint32_t rows, int64_t cols, uint8_t* q,
                                                    uint8_t* e) {
  const uint32_t nb = static_cast<uint32_t>(q8_ceil(cols, kQ8Block));
  const int64_t qp = q8_row_bytes(cols), ep = q8_exp_bytes(cols);
  const uint32_t total = rows * nb;  // below 2^31 (checked by the caller)
  const int lane = threadIdx.x & 15;
  // a workgroup's kU * 16 blocks are consecutive, and so is each step's 4 KiB
  const uint32_t b0 = blockIdx.x * (16 * kU) + (threadIdx.x >> 4);
  Chunk c[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const uint32_t b = b0 + u * 16;
    const uint32_t t = b / nb, k = b - t * nb;
    c[u] = b < total ? load8<DT, VEC>(x, t, static_cast<int64_t>(k) * kQ8Block + lane * 8, cols) : zero_chunk();
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const uint32_t b = b0 + u * 16;
    const uint32_t t = b / nb, k = b - t * nb;
    float v[8];
    chunk_to_f32<DT>(c[u], v);
    q8_quiet<DT>(v);
    const uint32_t byte = q8_exp_byte(q8_block_amax(v));
    if (b >= total) continue;
    *reinterpret_cast<uint2*>(q + static_cast<int64_t>(t) * qp + static_cast<int64_t>(k) * kQ8Block + lane * 8) =
        q8_encode8(v, q8_scale(byte));
    uint8_t* er = e + static_cast<int64_t>(t) * ep;
    if (lane == 0) er[k] = static_cast<uint8_t>(byte);
    if (k == nb - 1 && lane > 0 && k + lane < ep) er[k + lane] = 127;  // the exponent row's padding
  }
}

// One workgroup a tile: 128 rows of 16 chunks, eight chunks a thread in registers.
template <int DT, bool VEC>
__global__ __launch_bounds__(256) void q8_pack_tile(const void* W, int64_t out, int64_t in, uint32_t nb, uint8_t* q,
                                                    uint8_t* e) {
  __shared__ float wmax[4];
  const int64_t qp = q8_row_bytes(in), ep = q8_exp_bytes(in);
  const uint32_t ob = blockIdx.x / nb, ib = blockIdx.x - ob * nb;
  const int lane = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  const int64_t col = static_cast<int64_t>(ib) * kQ8Block + lane * 8;
  Chunk c[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int64_t row = static_cast<int64_t>(ob) * kQ8Block + u * 16 + r0;
    c[u] = row < out ? load8<DT, VEC>(W, row, col, in) : zero_chunk();
  }
  float a = 0.0f;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    float v[8];
    chunk_to_f32<DT>(c[u], v);
    q8_quiet<DT>(v);
    a = __builtin_fmaxf(a, q8_block_amax(v));
  }
#pragma unroll
  for (int d = 16; d < 64; d <<= 1) a = __builtin_fmaxf(a, __shfl_xor(a, d, 64));
  if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = a;
  __syncthreads();
  a = __builtin_fmaxf(__builtin_fmaxf(wmax[0], wmax[1]), __builtin_fmaxf(wmax[2], wmax[3]));
  const uint32_t byte = q8_exp_byte(a);
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const int64_t row = static_cast<int64_t>(ob) * kQ8Block + u * 16 + r0;
    float v[8];
    chunk_to_f32<DT>(c[u], v);
    q8_quiet<DT>(v);
    *reinterpret_cast<uint2*>(q + row * qp + col) = q8_encode8(v, q8_scale(byte));
  }
  uint8_t* er = e + static_cast<int64_t>(ob) * ep;
  if (threadIdx.x == 0) er[ib] = static_cast<uint8_t>(byte);
  if (ib == nb - 1 && threadIdx.x > 0 && ib + threadIdx.x < ep) er[ib + threadIdx.x] = 127;
}

template <int DT, bool VEC>
__global__ __launch_bounds__(256) void q8_unpack_k(const uint8_t* q, const uint8_t* e, uint32_t rows, int64_t cols,
                                                   int tile_shift, void* x) {
  using T16 = typename Dt<DT>::T;
  const uint32_t nb = static_cast<uint32_t>(q8_ceil(cols, kQ8Block));
  const int64_t qp = q8_row_bytes(cols), ep = q8_exp_bytes(cols);
  const uint32_t total = rows * nb;
  const int lane = threadIdx.x & 15;
  const uint32_t b0 = blockIdx.x * (16 * kU) + (threadIdx.x >> 4);
  uint2 w[kU];
  uint32_t byte[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const uint32_t b = b0 + u * 16;
    const uint32_t t = b / nb, k = b - t * nb;
    w[u] = uint2{0u, 0u};
    byte[u] = 127;
    if (b < total) {
      w[u] = *reinterpret_cast<const uint2*>(q + static_cast<int64_t>(t) * qp + static_cast<int64_t>(k) * kQ8Block +
                                             lane * 8);
      byte[u] = e[static_cast<int64_t>(t >> tile_shift) * ep + k];
    }
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const uint32_t b = b0 + u * 16;
    if (b >= total) continue;
    const uint32_t t = b / nb, k = b - t * nb;
    const int64_t col = static_cast<int64_t>(k) * kQ8Block + lane * 8;
    float f[8];
    q8_decode8(w[u], q8_scale(byte[u]), f);
    q8_hold<DT>(f);
    T16* p = static_cast<T16*>(x) + static_cast<int64_t>(t) * cols + col;
    if constexpr (VEC) {
      if (col < cols) *reinterpret_cast<Chunk*>(p) = f32_to_chunk<DT>(f);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col + i < cols) p[i] = Dt<DT>::from_f(f[i]);
    }
  }
}

template <class F>
void by_type(int dtype, bool vec, F f) {
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  if (dtype == 0)
    vec ? f(I0{}, std::true_type{}) : f(I0{}, std::false_type{});
  else
    vec ? f(I1{}, std::true_type{}) : f(I1{}, std::false_type{});
}

}  // namespace

hipError_t launch_q8_pack(const void* x, int64_t rows, int64_t cols, int dtype, bool vec, void* q, void* e,
                          hipStream_t stream) {
  const int64_t blocks = rows * q8_ceil(cols, kQ8Block);
  if (blocks == 0) return hipSuccess;
  by_type(dtype, vec, [&](auto dt, auto v) {
    hipLaunchKernelGGL((q8_pack_rows<decltype(dt)::value, decltype(v)::value>),
                       dim3(static_cast<unsigned>(q8_ceil(blocks, 16 * kU))), dim3(256), 0, stream, x,
                       static_cast<uint32_t>(rows), cols, static_cast<uint8_t*>(q), static_cast<uint8_t*>(e));
  });
  return hipGetLastError();
}

hipError_t launch_q8_pack_tiles(const void* W, int64_t out, int64_t in, int dtype, bool vec, void* q, void* e,
                                hipStream_t stream) {
  const int64_t nb = q8_ceil(in, kQ8Block), tiles = nb * q8_ceil(out, kQ8Block);
  if (tiles == 0) return hipSuccess;
  by_type(dtype, vec, [&](auto dt, auto v) {
    hipLaunchKernelGGL((q8_pack_tile<decltype(dt)::value, decltype(v)::value>), dim3(static_cast<unsigned>(tiles)),
                       dim3(256), 0, stream, W, out, in, static_cast<uint32_t>(nb), static_cast<uint8_t*>(q),
                       static_cast<uint8_t*>(e));
  });
  return hipGetLastError();
}

hipError_t launch_q8_unpack(const void* q, const void* e, int64_t rows, int64_t cols, bool tiles, int dtype, bool vec,
                            void* x, hipStream_t stream) {
  const int64_t blocks = rows * q8_ceil(cols, kQ8Block);
  if (blocks == 0) return hipSuccess;
  by_type(dtype, vec, [&](auto dt, auto v) {
    hipLaunchKernelGGL((q8_unpack_k<decltype(dt)::value, decltype(v)::value>),
                       dim3(static_cast<unsigned>(q8_ceil(blocks, 16 * kU))), dim3(256), 0, stream,
                       static_cast<const uint8_t*>(q), static_cast<const uint8_t*>(e), static_cast<uint32_t>(rows),
                       cols, tiles ? 7 : 0, x);
  });
  return hipGetLastError();
}

}  // namespace dora
