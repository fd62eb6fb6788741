// What the C entry points share on the host: the calling thread's error
// message, status helpers, and the argument checks.  Nothing here allocates or
// throws.
#pragma once

#include <hip/hip_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/dora.h"

namespace dora {
namespace abi {

inline thread_local char g_err[512] = "";

inline int fail(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_err, sizeof(g_err), fmt, ap);
  va_end(ap);
  return status;
}

inline int ok() {
  g_err[0] = '\0';
  return DORA_OK;
}

inline int hip_status(hipError_t e, const char* what) {
  if (e == hipSuccess) return ok();
  return fail(DORA_HIP_ERROR, "%s: %s", what, hipGetErrorString(e));
}

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned(p, 16); }

// Two byte ranges [p, p + n) and [q, q + m) that overlap without being the same buffer.
inline bool partial_overlap(const void* p, size_t n, const void* q, size_t m) {
  if (!p || !q || n == 0 || m == 0) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  if (a == b && n == m) return false;
  return a < b + m && b < a + n;
}

inline bool any_overlap(const void* p, size_t n, const void* q, size_t m) {
  if (!p || !q || n == 0 || m == 0) return false;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + m && b < a + n;
}

inline bool valid_dtype(int dtype) { return dtype == DORA_BF16 || dtype == DORA_F16; }

// A byte range of a call, for the overlap checks.
struct Range {
  const void* p;
  size_t n;
};

// True when an output overlaps an input or another output.
template <int NO, int NI>
inline bool outputs_overlap(const Range (&outs)[NO], const Range (&ins)[NI]) {
  for (int o = 0; o < NO; ++o) {
    for (int i = 0; i < NI; ++i)
      if (any_overlap(outs[o].p, outs[o].n, ins[i].p, ins[i].n)) return true;
    for (int q = o + 1; q < NO; ++q)
      if (any_overlap(outs[o].p, outs[o].n, outs[q].p, outs[q].n)) return true;
  }
  return false;
}

}  // namespace abi
}  // namespace dora
