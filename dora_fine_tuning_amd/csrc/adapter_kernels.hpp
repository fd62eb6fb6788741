// Launch interface of the operators that sort tokens by adapter and exchange rows
// between the tokens' order and the adapters'.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dora {

// The sort's counters, one of each wave for each adapter, lie in 64 KB of LDS.
constexpr int64_t kMaxAdapters = 1000;

// ids: int64 (id_bytes 8) or int32 (4), N of them.
struct AdapterSortArgs {
  const void* ids;
  int id_bytes;
  int64_t N, n;
  int32_t *order, *place, *bounds;
  void* ws;
  hipStream_t stream;
};
size_t adapter_sort_workspace_bytes(int64_t N, int64_t n);
hipError_t launch_adapter_sort(const AdapterSortArgs& a);

// T tokens of k slots, rows of D elements; pointers that an operator does not
// take, or that the caller leaves out, are null.
struct AdapterRowsArgs {
  const void *x, *rows, *base;
  const float* weights;
  const int32_t* place;
  int64_t T, k, D;
  int dtype;
  bool vec;  // D % 8 == 0, 16-byte aligned rows
  void *y, *d_rows;
  float* d_weights;
  hipStream_t stream;
};
constexpr int kAdapterRowThreads = 256;
int64_t adapter_rows_grid(int64_t T, int64_t D);  // workgroups
hipError_t launch_adapter_gather(const AdapterRowsArgs& a);       // x, place -> y [T k x D]
hipError_t launch_adapter_combine(const AdapterRowsArgs& a);      // rows, weights, place, base -> y [T x D]
hipError_t launch_adapter_combine_bwd(const AdapterRowsArgs& a);  // x = dy, rows, weights, place -> d_rows, d_weights

}  // namespace dora
