// fm_seqs.cuh -- what the attention kernels over requests of different lengths share: the key
// tiles that a unit sees, and where a key's row lies.
#pragma once

#include "fm_internal.h"

namespace fm {
namespace {

struct TileRange {
  int a, e;  // key tiles [a, e) hold every key that some row of the unit sees; hi: one past the last such key
  int hi;
};
// Unit of `nt` tokens whose first stands at position pos0 among the kv keys of its request
// (negative when there are more queries than keys).  Token at position p sees keys j <= p
// (causal), j > p - window (window > 0).
__device__ __forceinline__ TileRange unit_tiles(int pos0, int nt, int kv, int bk, int causal, int window) {
  const int hi = causal ? max(0, min(kv, pos0 + nt)) : kv;
  const int lo = window > 0 ? max(0, pos0 - window + 1) : 0;
  TileRange r;
  r.hi = hi;
  r.a = lo / bk;
  r.e = hi > lo ? (hi + bk - 1) / bk : r.a;
  return r;
}

// Keys [lo, hi) that the token at position p sees.
__device__ __forceinline__ void seen_keys(int p, int kv, int causal, int window, int &lo, int &hi) {
  hi = causal ? min(kv, p + 1) : kv;
  lo = window > 0 ? p - window + 1 : 0;
}

__device__ __forceinline__ void report_bad_page(unsigned int *err, int request, int position, int page) {
  if (err && atomicCAS(err, 0u, (unsigned)kDevErrPage) == 0u) {
    err[1] = (unsigned)request;
    err[2] = (unsigned)position;
    err[3] = (unsigned)page;
  }
}

}  // namespace
}  // namespace fm
