// Tokens sorted by adapter, and rows exchanged between the tokens' order and the
// adapters', for gfx950.
//
// A batch's token t has k slots, each with the number of an adapter in [0, n), or
// none.  Slots t * k + j are sorted by adapter, stably, those without one behind
// them all: place[t, j] = p says that the slot's row is p, the complement ~p that
// it is p and has no adapter.  A row belongs to exactly one slot.
//
//   gather       rows[p] = x[t]                         (0 without an adapter)
//   combine      y[t] = base[t] + sum_j w[t, j] rows[place[t, j]]
//   its backward d_rows[p] = w[t, j] dy[t],  d_w[t, j] = <dy[t], rows[p]>
//
// gather's backward is combine without weights or base.  All go by tokens: the
// threads of a token read or write its row and its k rows, so that no sum needs an
// atomic, and every row is written, those without an adapter as zeros.  Gather and
// combine read each row once; combine's backward takes the slots in turn and reads
// the row of dy for each, after the first from the caches (the bytes of the rates
// below count it once).
//
// HBM bounds the rows (8192 tokens of 2 slots, rows of 8192 in bf16: gather 77 us, 5.2
// TB/s; combine with base and weights 100, 5.3; its backward 135, 5.0; one slot and
// rows of 4096: 22, 32 and 33, 6.0 TB/s), and latency everything small (37 tokens:
// 2.7 and 3.3).
#include <algorithm>

#include "adapter_kernels.hpp"
#include "dora_common.hpp"
#include "q4_common.hpp"

namespace dora {

namespace {

// ------------------------------------------------------------------ sorting
//
// A counting sort.  A workgroup takes a range of slots, each of its waves a
// contiguous part of it.  The waves count their keys in LDS; an adapter's first
// row is the slots of smaller adapters, and a wave's first row of it the slots
// of that adapter in earlier workgroups (from a table that a first launch
// leaves) and earlier waves.  Then 64 slots at a time: lanes with equal keys find
// each other by ballots over the keys' bits, the lowest of them moves the
// counter, and a lane's rank is the number of such lanes below it: the order is that
// of the slots, whichever wave is first.  Latency bounds it: 3.3 us for 37 slots, 6.3
// for 4096, 8.3 for 20480 (two launches from 4097 on), 12 for 262144, 23 for a million.
constexpr int kSortWaves = 16, kSortThreads = 64 * kSortWaves;
constexpr int kSortRounds = 4;  // of 64 slots a wave, whose keys stay in registers

struct SortArgs {
  const void* ids;
  int wide;  // ids are 64-bit
  int64_t N;
  int n;
  int rounds;  // of 64 slots a wave
  int chunks;
  int bits;  // of a key
  int32_t *order, *place, *bounds;
  int32_t* table;  // [chunks x (n + 1)]
};

__device__ inline int key_of(const SortArgs& a, int64_t slot) {
  if (a.wide) {
    const int64_t v = static_cast<const int64_t*>(a.ids)[slot];
    return v >= 0 && v < a.n ? static_cast<int>(v) : a.n;
  }
  const int32_t v = static_cast<const int32_t*>(a.ids)[slot];
  return v >= 0 && v < a.n ? v : a.n;
}

// The wave's keys of its first rounds, -1 past the last slot, and the counts of the
// workgroup's waves: cnt[wave * (n + 1) + key].
__device__ inline void count_keys(const SortArgs& a, int32_t* cnt, int64_t first, int wave, int lane,
                                  int (&mine)[kSortRounds]) {
  const int keys = a.n + 1;
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t slot = first + r * 64 + lane;
    mine[r] = r < a.rounds && slot < a.N ? key_of(a, slot) : -1;
  }
  for (int i = threadIdx.x; i < keys * kSortWaves; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r)
    if (mine[r] >= 0) atomicAdd(&cnt[wave * keys + mine[r]], 1);
  for (int r = kSortRounds; r < a.rounds; ++r) {
    const int64_t slot = first + r * 64 + lane;
    if (slot < a.N) atomicAdd(&cnt[wave * keys + key_of(a, slot)], 1);
  }
  __syncthreads();
}

__device__ inline int64_t first_slot(const SortArgs& a, int wave) {
  return (static_cast<int64_t>(blockIdx.x) * kSortWaves + wave) * a.rounds * 64;
}

__global__ __launch_bounds__(kSortThreads) void adapter_count(SortArgs a) {
  extern __shared__ int32_t cnt[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, keys = a.n + 1;
  int mine[kSortRounds];
  count_keys(a, cnt, first_slot(a, wave), wave, lane, mine);
  for (int key = threadIdx.x; key < keys; key += kSortThreads) {
    int32_t s = 0;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) s += cnt[w * keys + key];
    a.table[static_cast<int64_t>(blockIdx.x) * keys + key] = s;
  }
}

__global__ __launch_bounds__(kSortThreads) void adapter_sort_k(SortArgs a) {
  extern __shared__ int32_t cnt[];
  __shared__ int32_t sums[kSortWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, keys = a.n + 1;
  const int64_t first = first_slot(a, wave);
  int mine[kSortRounds];
  count_keys(a, cnt, first, wave, lane, mine);

  // a key a thread (n <= 1000, and the slots without an adapter): its slots in the
  // waves, in all, and in earlier workgroups
  const int key = threadIdx.x;
  int32_t of_wave[kSortWaves], total = 0, before = 0;
  if (key < keys) {
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) of_wave[w] = cnt[w * keys + key];
    if (a.chunks == 1) {
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) total += of_wave[w];
    } else {
#pragma unroll 8
      for (int c = 0; c < a.chunks; ++c) {
        if (c == static_cast<int>(blockIdx.x)) before = total;
        total += a.table[static_cast<int64_t>(c) * keys + key];
      }
    }
  }
  // the first row of each: an exclusive sum over the threads
  int32_t upto = total;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int32_t v = __shfl_up(upto, d, 64);
    if (lane >= d) upto += v;
  }
  if (lane == 63) sums[wave] = upto;
  __syncthreads();
  int32_t lower = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) lower += w < wave ? sums[w] : 0;
  const int32_t start = lower + upto - total;
  if (key < keys) {
    if (blockIdx.x == 0) a.bounds[key] = start;  // the last key's start is the end of the adapters' rows
    // the counters become the next row of each key
    int32_t row = start + before;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      cnt[w * keys + key] = row;
      row += of_wave[w];
    }
  }
  __syncthreads();

  const uint64_t below = (uint64_t(1) << lane) - 1;
  auto place64 = [&](int r, int kk) {
    const bool on = kk >= 0;
    uint64_t same = __ballot(on);
    for (int b = 0; b < a.bits; ++b) {
      const uint64_t set = __ballot((kk >> b) & 1);
      same &= ((kk >> b) & 1) ? set : ~set;
    }
    if (on) {
      const int lead = __builtin_ctzll(same);
      int32_t row = 0;
      if (lane == lead) row = atomicAdd(&cnt[wave * keys + kk], __popcll(same));
      row = __shfl(row, lead, 64) + __popcll(same & below);
      const bool has = kk < a.n;
      const int64_t slot = first + r * 64 + lane;
      const int32_t s32 = static_cast<int32_t>(slot);
      a.order[row] = has ? s32 : ~s32;
      a.place[slot] = has ? row : ~row;
    }
  };
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r)
    if (r < a.rounds) place64(r, mine[r]);
  for (int r = kSortRounds; r < a.rounds; ++r) {
    const int64_t slot = first + r * 64 + lane;
    place64(r, slot < a.N ? key_of(a, slot) : -1);
  }
}

// Up to 4096 slots are one workgroup's, in one launch.  More are spread over up to 64
// with one to four rounds each, and beyond over 256, whose table each of them reads.
int sort_rounds(int64_t N) {
  if (N <= kSortThreads * kSortRounds) return static_cast<int>(std::max<int64_t>(1, q4_ceil(N, kSortThreads)));
  if (N <= 64 * kSortThreads * kSortRounds) return static_cast<int>(q4_ceil(N, 64 * kSortThreads));
  return static_cast<int>(std::max<int64_t>(kSortRounds, q4_ceil(N, 256 * kSortThreads)));
}
int64_t sort_chunks(int64_t N) { return std::max<int64_t>(1, q4_ceil(N, int64_t(kSortThreads) * sort_rounds(N))); }

// ------------------------------------------------------------------ rows
//
// A token's row is shared by `span` threads (a power of two up to 256), each
// taking chunks of 8 elements, kU of them at a time.
constexpr int kRowThreads = kAdapterRowThreads, kU = 4;

struct RowsArgs {
  const void *x, *rows, *base;
  const float* w;
  const int32_t* place;
  int64_t T, R, D;  // R = T k rows
  int k, span;
  void *y, *d_rows;
  float* d_w;
};

template <int DT, bool VEC>
__device__ inline Chunk load_chunk(const void* p, int64_t row, int64_t c, int64_t D) {
  using T16 = typename Dt<DT>::T;
  const T16* s = static_cast<const T16*>(p) + row * D + c;
  if constexpr (VEC) {
    return *reinterpret_cast<const Chunk*>(s);
  } else {
    typename Dt<DT>::V8 v;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < D ? s[j] : static_cast<T16>(0.0f);
    return __builtin_bit_cast(Chunk, v);
  }
}
template <int DT, bool VEC>
__device__ inline void store_chunk(void* p, int64_t row, int64_t c, int64_t D, const Chunk& v) {
  using T16 = typename Dt<DT>::T;
  T16* d = static_cast<T16*>(p) + row * D + c;
  if constexpr (VEC) {
    *reinterpret_cast<Chunk*>(d) = v;
  } else {
    const auto e = __builtin_bit_cast(typename Dt<DT>::V8, v);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < D) d[j] = e[j];
  }
}

template <int DT, bool VEC>
__global__ __launch_bounds__(kRowThreads) void adapter_gather_k(RowsArgs a) {
  const int me = threadIdx.x & (a.span - 1);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRowThreads / a.span) + threadIdx.x / a.span;
  if (t >= a.T) return;
  const int64_t step = static_cast<int64_t>(a.span) * 8;
  for (int64_t c0 = me * 8; c0 < a.D; c0 += kU * step) {
    Chunk v[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (c0 + u * step < a.D) v[u] = load_chunk<DT, VEC>(a.x, t, c0 + u * step, a.D);
    for (int j = 0; j < a.k; ++j) {
      const int32_t p = a.place[t * a.k + j];
      const int64_t row = p < 0 ? ~p : p;
      if (row >= a.R) continue;
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (c0 + u * step < a.D)
          store_chunk<DT, VEC>(a.y, row, c0 + u * step, a.D, p < 0 ? zero_chunk() : v[u]);
    }
  }
}

template <int DT, bool VEC>
__global__ __launch_bounds__(kRowThreads) void adapter_combine_k(RowsArgs a) {
  const int me = threadIdx.x & (a.span - 1);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRowThreads / a.span) + threadIdx.x / a.span;
  if (t >= a.T) return;
  const int64_t step = static_cast<int64_t>(a.span) * 8;
  for (int64_t c0 = me * 8; c0 < a.D; c0 += kU * step) {
    float s[kU][8];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      Chunk b = zero_chunk();
      if (a.base && c0 + u * step < a.D) b = load_chunk<DT, VEC>(a.base, t, c0 + u * step, a.D);
      chunk_to_f32<DT>(b, s[u]);
    }
    for (int j0 = 0; j0 < a.k; j0 += 2) {  // two slots' loads at a time, added in order
      Chunk v[2][kU];
      float w[2];
      bool on[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t slot = t * a.k + j0 + h;
        const int32_t p = j0 + h < a.k ? a.place[slot] : -1;
        on[h] = p >= 0 && p < a.R;
        w[h] = on[h] && a.w ? a.w[slot] : 1.0f;
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (on[h] && c0 + u * step < a.D) v[h][u] = load_chunk<DT, VEC>(a.rows, p, c0 + u * step, a.D);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!on[h]) continue;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          if (c0 + u * step >= a.D) break;
          float f[8];
          chunk_to_f32<DT>(v[h][u], f);
#pragma unroll
          for (int i = 0; i < 8; ++i) s[u][i] = __builtin_fmaf(w[h], f[i], s[u][i]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (c0 + u * step < a.D) store_chunk<DT, VEC>(a.y, t, c0 + u * step, a.D, f32_to_chunk<DT>(s[u]));
  }
}

// Both gradients in one pass over dy and the rows.  Every thread of the workgroup
// reaches the sums over the token's threads.
template <int DT, bool VEC>
__global__ __launch_bounds__(kRowThreads) void adapter_combine_bwd_k(RowsArgs a) {
  __shared__ float part[kRowThreads / 64];
  const int me = threadIdx.x & (a.span - 1);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kRowThreads / a.span) + threadIdx.x / a.span;
  const int64_t step = static_cast<int64_t>(a.span) * 8;
  const int64_t D = t < a.T ? a.D : 0;
  for (int j = 0; j < a.k; ++j) {
    const int32_t p = t < a.T ? a.place[t * a.k + j] : 0;
    const int64_t row = p < 0 ? ~p : p;
    const bool in = row < a.R, has = in && p >= 0;
    const float w = a.w && t < a.T ? a.w[t * a.k + j] : 1.0f;
    float dot = 0.0f;
    for (int64_t c0 = me * 8; c0 < D; c0 += kU * step) {
      Chunk d[kU], v[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (c0 + u * step >= D) break;
        d[u] = has ? load_chunk<DT, VEC>(a.x, t, c0 + u * step, D) : zero_chunk();
        if (a.d_w) v[u] = has ? load_chunk<DT, VEC>(a.rows, row, c0 + u * step, D) : zero_chunk();
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        if (c0 + u * step >= D) break;
        float f[8];
        chunk_to_f32<DT>(d[u], f);
        if (a.d_w) {
          float r[8];
          chunk_to_f32<DT>(v[u], r);
#pragma unroll
          for (int i = 0; i < 8; ++i) dot = __builtin_fmaf(f[i], r[i], dot);
        }
        if (a.d_rows && in) {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] *= w;
          store_chunk<DT, VEC>(a.d_rows, row, c0 + u * step, D, has ? f32_to_chunk<DT>(f) : zero_chunk());
        }
      }
    }
    if (a.d_w) {
      for (int d = std::min(a.span, 64) >> 1; d > 0; d >>= 1) dot += __shfl_xor(dot, d, 64);
      if (a.span > 64) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
        __syncthreads();
        const int w0 = (threadIdx.x & ~(a.span - 1)) >> 6;
        dot = part[w0] + part[w0 + 1];
        if (a.span > 128) dot += part[w0 + 2] + part[w0 + 3];
      }
      if (me == 0 && t < a.T) a.d_w[t * a.k + j] = dot;
    }
  }
}

// Threads a token: as many as leave each at most kU chunks, 256 at most.
int row_span(int64_t D) {
  int s = 1;
  while (s < kRowThreads && static_cast<int64_t>(s) * 8 * kU < D) s *= 2;
  return s;
}

// The kernels of an operator by dtype and by 16-byte rows.
using RowsKernel = void (*)(RowsArgs);
hipError_t launch_rows(const AdapterRowsArgs& a, const RowsKernel (&kernels)[2][2]) {
  const RowsArgs r{a.x, a.rows, a.base, a.weights, a.place, a.T, a.T * a.k, a.D, static_cast<int>(a.k), row_span(a.D),
                   a.y, a.d_rows, a.d_weights};
  hipLaunchKernelGGL(kernels[a.dtype][a.vec ? 1 : 0], dim3(static_cast<unsigned>(adapter_rows_grid(a.T, a.D))),
                     dim3(kRowThreads), 0, a.stream, r);
  return hipGetLastError();
}

}  // namespace

size_t adapter_sort_workspace_bytes(int64_t N, int64_t n) {
  const int64_t c = sort_chunks(N);
  return c > 1 ? static_cast<size_t>(c) * (n + 1) * 4 : 0;
}

hipError_t launch_adapter_sort(const AdapterSortArgs& p) {
  SortArgs a{};
  a.ids = p.ids;
  a.wide = p.id_bytes == 8;
  a.N = p.N;
  a.n = static_cast<int>(p.n);
  a.rounds = sort_rounds(p.N);
  a.chunks = static_cast<int>(sort_chunks(p.N));
  while ((1 << a.bits) < a.n + 1) ++a.bits;
  a.order = p.order;
  a.place = p.place;
  a.bounds = p.bounds;
  a.table = static_cast<int32_t*>(p.ws);
  const dim3 grid(a.chunks), block(kSortThreads);
  const size_t lds = static_cast<size_t>(kSortWaves) * (a.n + 1) * 4;  // 64064 bytes at most
  if (a.chunks > 1) {
    hipLaunchKernelGGL(adapter_count, grid, block, lds, p.stream, a);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(adapter_sort_k, grid, block, lds, p.stream, a);
  return hipGetLastError();
}

int64_t adapter_rows_grid(int64_t T, int64_t D) { return q4_ceil(T, kRowThreads / row_span(D)); }

hipError_t launch_adapter_gather(const AdapterRowsArgs& a) {
  return launch_rows(a, {{adapter_gather_k<0, false>, adapter_gather_k<0, true>},
                         {adapter_gather_k<1, false>, adapter_gather_k<1, true>}});
}
hipError_t launch_adapter_combine(const AdapterRowsArgs& a) {
  return launch_rows(a, {{adapter_combine_k<0, false>, adapter_combine_k<0, true>},
                         {adapter_combine_k<1, false>, adapter_combine_k<1, true>}});
}
hipError_t launch_adapter_combine_bwd(const AdapterRowsArgs& a) {
  return launch_rows(a, {{adapter_combine_bwd_k<0, false>, adapter_combine_bwd_k<0, true>},
                         {adapter_combine_bwd_k<1, false>, adapter_combine_bwd_k<1, true>}});
}

}  // namespace dora
