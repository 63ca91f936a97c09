// fm_tree.cuh -- what the kernels on trees of drafted tokens share.
#pragma once

#include "fm_internal.h"

namespace fm {
namespace {

__device__ __forceinline__ void report(unsigned int *err, unsigned int code, unsigned int a, unsigned int b, unsigned int c,
                                       unsigned int d) {
  if (err && atomicCAS(err, 0u, code) == 0u) {
    err[1] = a;
    err[2] = b;
    err[3] = c;
    err[4] = d;
  }
}

// Rows [first, first + count) of request b, clamped to T rows; starts that do not fit are reported.
struct Rows {
  int first, count;
};
__device__ __forceinline__ Rows rows_of(const int32_t *cu, int b, int64_t T, unsigned int *err) {
  const int r0 = cu[b], r1 = cu[b + 1];
  Rows r;
  r.first = (int)max((int64_t)0, min((int64_t)r0, T));
  r.count = (int)max((int64_t)r.first, min((int64_t)r1, T)) - r.first;
  if (r.first != r0 || r.first + r.count != r1) report(err, kDevErrLength, (unsigned)b, (unsigned)r0, (unsigned)r1, 0u);
  return r;
}

}  // namespace
}  // namespace fm
