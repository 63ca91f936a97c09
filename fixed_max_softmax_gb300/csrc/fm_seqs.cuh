// fm_seqs.cuh -- what the attention kernels over requests of different lengths share: the key
// tiles that a unit sees, and where a key's row lies.
#pragma once

#include <limits.h>

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

// Lengths of a call's requests (device arrays and the tensors' extents).
struct SeqsLens {
  const int32_t *cu_q, *cu_k, *kv_len;
  int64_t T, Tk, cap_keys;  // cap_keys: keys that a row of the page table can hold
  int paged;
};
struct Request {
  int q0, q, kv, k0;  // first query row, queries, keys, first key row (packed)
  bool back;          // its starts run backwards: requests overlap, and nothing of the call is computed
};
// Request b, clamped to the tensors; what does not fit is reported when `err` is given.
__device__ __forceinline__ Request request_of(const SeqsLens &s, int b, unsigned int *err) {
  const int r0 = s.cu_q[b], r1 = s.cu_q[b + 1];
  Request r;
  r.q0 = (int)max((int64_t)0, min((int64_t)r0, s.T));
  r.q = (int)max((int64_t)r.q0, min((int64_t)r1, s.T)) - r.q0;
  r.back = r1 < r0;
  bool bad = r.q0 != r0 || r.q0 + r.q != r1;
  r.k0 = 0;
  if (s.paged) {
    const int x = s.kv_len[b];
    r.kv = (int)max((int64_t)0, min((int64_t)x, s.cap_keys));
    bad |= r.kv != x;
  } else {
    const int x0 = s.cu_k[b], x1 = s.cu_k[b + 1];
    r.k0 = (int)max((int64_t)0, min((int64_t)x0, s.Tk));
    r.kv = (int)max((int64_t)r.k0, min((int64_t)x1, s.Tk)) - r.k0;
    bad |= r.k0 != x0 || r.k0 + r.kv != x1;
  }
  if (bad && err && atomicCAS(err, 0u, (unsigned)kDevErrLength) == 0u) {
    err[1] = (unsigned)b;
    err[2] = (unsigned)r0;
    err[3] = (unsigned)r1;
    err[4] = (unsigned)r.kv;
  }
  return r;
}
inline SeqsLens seqs_lens(const SeqsArgs &a) {
  SeqsLens s;
  s.cu_q = a.cu_q;
  s.cu_k = a.cu_k;
  s.kv_len = a.kv_len;
  s.T = a.q.S;
  s.Tk = a.paged ? 0 : a.k.S;
  s.cap_keys = a.paged ? a.table_width * a.k.S : 0;
  if (s.cap_keys > ((int64_t)1 << 30)) s.cap_keys = (int64_t)1 << 30;
  s.paged = a.paged;
  return s;
}

// Keys [lo, hi) that the token at position p sees.
__device__ __forceinline__ void seen_keys(int p, int kv, int causal, int window, int &lo, int &hi) {
  hi = causal ? min(kv, p + 1) : kv;
  lo = window > 0 ? p - window + 1 : 0;
}

// Trees of drafted tokens.  Of its request's new tokens a row sees those whose bits are set in its mask
// row, bit 0 being the first; earlier keys it sees all.  Causal requests (prompt chunks of more tokens
// than a mask row has bits) get a base that no key reaches.
struct TreeRow {
  int base;              // the request's first new token among its keys
  int words;             // of the mask row (0: no row)
  const uint32_t *bits;
};
__device__ __forceinline__ TreeRow tree_row(const SeqsLens &s, const uint32_t *mask, int words, int64_t stride, int b, int kv,
                                            int64_t row, bool ok) {
  const int q0 = (int)max((int64_t)0, min((int64_t)s.cu_q[b], s.T));
  const int q = (int)max((int64_t)q0, min((int64_t)s.cu_q[b + 1], s.T)) - q0;
  TreeRow r;
  r.base = q <= 32 * words ? kv - q : INT_MAX;
  r.words = ok ? words : 0;
  r.bits = mask + row * stride;
  return r;
}
// Bits n0 .. n0 + 31 of a mask row; the keys before its bit 0 are all seen, those behind its last word not.
__device__ __forceinline__ uint32_t tree_bits(const uint32_t *bits, int words, int n0) {
  const int w = n0 >> 5;
  const uint32_t lo = w < 0 ? 0xffffffffu : (w < words ? bits[w] : 0u);
  const uint32_t hi = w + 1 < 0 ? 0xffffffffu : (w + 1 < words ? bits[w + 1] : 0u);
  return __funnelshift_r(lo, hi, (uint32_t)n0 & 31u);
}
// Is the key at `key` seen?
__device__ __forceinline__ bool tree_sees(const TreeRow &r, int key) {
  const int n = key - r.base;
  return n < 0 || ((n >> 5) < r.words && ((r.bits[n >> 5] >> (n & 31)) & 1u));
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
