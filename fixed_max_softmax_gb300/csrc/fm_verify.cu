// fm_verify.cu -- verification of a tree of drafted tokens against the target's probabilities.
//
// The walk begins at node 0 and tries a node's children in order.  With p the target's row after the
// node that the walk stands at, q the draft's, and A = 0, S = 1 when it arrives there:
//   child of token x and number u is kept  <=>  u q(x) S < max(p(x) - A q(x), 0)
//   not kept:  A += S,  S = sum_y max(p(y) - A q(y), 0)      (S = 0: A = 0, S = 1)
// which is rejection sampling: what is left of p after k children drawn from q were refused is
// R_k = max(R_{k-1} - S_{k-1} q, 0), R_0 = p, S_k its sum, and since q >= 0 these nest into
// R_k = max(p - (S_0 + .. + S_{k-1}) q, 0): one number A says what is left of every token, and nothing
// of a vocabulary's length is stored.  Of children that were chosen and not drawn (no draft row) one
// is kept if u S < p(x); else S -= p(x) and p(x) := 0.  Where the walk ends the next token is the least
// x with sum_{y <= x} R(y) > u_last sum_y R(y).
//
// A cluster of up to 8 CTAs a request.  Its first CTA gathers the nodes' parents, tokens, numbers and
// the p and q that their tests compare into every CTA's shared memory; from there the first warp of each
// CTA walks, all alike, and the CTAs meet only to sum what is left over the vocabulary, once a
// refused child and once at the end: each sums an even part of the row, and the parts' sums go to every
// CTA's shared memory.  A walk without a refusal reads one row of the vocabulary in all.
// Sums and tests are compared with random numbers, and a sum that is off by 2^-24 would pick another token
// than the definition does at every border that the number falls next to.  All of it is done in pairs of fp32
// numbers, a value and its error.  With u = 2^-24: of p - A q the error is at most u (p + 2 A q), and its two roundings
// 4 u^2 (p + A q).  A two-sum is exact, and what it lost, at most u of the sum so far, is added to the sum's
// error, which after N additions of total X, the elements' M = sum (p + 2 A q), is at most u (N X + M): its N
// roundings are at most (N^2 + N) u^2 M together.  N is V / 1024 + 20 where a request has one CTA; the
// roundings have either sign, and rows of softmaxes come out to 2^-48 up to 2^21 tokens, 2^-44 at 2^24.  An SM
// adds two 64-bit numbers a clock, and one takes
// some hundred clocks, a pair's addition a dozen fp32 operations (64 chains over 128,000 tokens: 152 us with
// 64-bit sums, 98 with pairs for the elements and 64 bits in every warp's tests, 29 with 64 bits in one warp of a
// CTA, 28 without any; 22 with two elements to an instruction).
// Bound by latency: at that size the row's sum takes 8 us, HBM's rate for its 65 MB, and the way to it and on
// (nodes, tests, the CTAs' meeting, the search for the border) as long again; a refusal at a row in L2 some 2 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <limits.h>
#include <math.h>

#include "fm_tree.cuh"

namespace fm {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32, kMostCtas = 8;

__device__ __forceinline__ uint32_t smem_at(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {  // the same address in another CTA of the cluster
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void put_remote(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ float as_f32(float x) { return x; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float as_f32(__half x) { return __half2float(x); }
// A probability: what is negative, infinite or no number counts as 0 (by its bits: all of these lie at or
// above infinity's).
__device__ __forceinline__ float some(float x) { return __float_as_uint(x) < 0x7f800000u ? x : 0.f; }

// Two fp32 lanes in one 64-bit register, added and multiplied in one instruction.
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_split(uint64_t v, float &lo, float &hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_sub(uint64_t a, uint64_t b) {  // a - b, rounded once
  return f2_fma(b, 0xbf800000bf800000ull, a);
}

// x + e, e the error of x: a pair of fp32 numbers holds what a sum in fp32 would lose.
struct Pair {
  float x, e;
};

struct Shared {
  int parent[FM_MAX_NODES], token[FM_MAX_NODES];  // token -1: outside the vocabulary
  float u[FM_MAX_NODES], p[FM_MAX_NODES], q[FM_MAX_NODES];
  int first, nodes;             // row of node 0, nodes (-1: not verified) and the last random number, as the first CTA read them
  float u_last;
  int refused[FM_MAX_NODES];    // tokens taken out of p (children that were chosen)
  Pair part[2][kMostCtas * kWarps];  // the sums of all CTAs' warps, of alternate passes
  Pair upto[32];                // the first warp's prefix sums over them
  Pair warp[kWarps];            // this CTA's warps' sums of a part
  // what the first warp has the others do: sum the row after node `cur` (A, n_refused tokens taken out),
  // or look for the border in the blocks [part0, part1) of it, or nothing more
  int what, cur, n_refused, part0, part1;
  Pair A;
};
enum : int { kSum, kFind, kDone };

// A row of one model in blocks of 16 bytes, block 0 beginning `shift` elements before the row: element `e`
// of block b is element b * VEC - shift + e of the row.  A target's row has the shift that puts its blocks on
// 16-byte boundaries; the draft's row is cut like it, and its blocks may lie anywhere: off a boundary they are
// read by elements (64 chains over 128,000 tokens fp32 19.3 -> 21.3 us, bf16 20.6 -> 25.1).
template <typename E>
struct Row {
  static constexpr int VEC = 16 / (int)sizeof(E);
  const E *at;  // of block 0
  int shift, V;
  int full0;             // the blocks that one load takes: on a boundary, and inside the row
  unsigned full;

  __device__ __forceinline__ Row(const void *base, int64_t stride, int64_t row, int V_, int shift_ = -1) : V(V_) {
    const E *p = reinterpret_cast<const E *>(base) + row * stride;
    const int own = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(E));
    shift = shift_ < 0 ? own : shift_;
    at = p - shift;
    full0 = shift > 0 ? 1 : 0;
    full = own == shift ? (unsigned)max((V + shift) / VEC - full0, 0) : 0u;
  }
  __device__ __forceinline__ int blocks() const { return (V + shift + VEC - 1) / VEC; }
  __device__ __forceinline__ uint4 load(int b) const {
    if ((unsigned)(b - full0) < full) return *reinterpret_cast<const uint4 *>(at + b * VEC);
    const int i = b * VEC - shift;  // in the row
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    E *e = reinterpret_cast<E *>(&w);
#pragma unroll
    for (int j = 0; j < VEC; ++j)
      if (i + j >= 0 && i + j < V) e[j] = at[b * VEC + j];
    return w;
  }
};

// The pair a + b: s = a + b rounded, and exactly what that lost (Knuth's two-sum).
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), bb = __fadd_rn(s, -a);
  return {s, __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -bb)), __fadd_rn(b, -bb))};
}
__device__ __forceinline__ void add(Pair &sum, Pair v) {
  const Pair s = two_sum(sum.x, v.x);
  sum.x = s.x;
  sum.e = __fadd_rn(sum.e, __fadd_rn(s.e, v.e));
}
__device__ __forceinline__ bool positive(Pair v) { return __fadd_rn(v.x, v.e) > 0.f; }
__device__ __forceinline__ bool less(Pair a, Pair b) {
  Pair d = two_sum(b.x, -a.x);
  d.e = __fadd_rn(d.e, __fadd_rn(b.e, -a.e));
  return positive(d);
}
__device__ __forceinline__ Pair times(Pair a, float b) {
  const float m = __fmul_rn(a.x, b);
  return {m, __fmaf_rn(a.e, b, __fmaf_rn(a.x, b, -m))};
}
__device__ __forceinline__ Pair shuffle(Pair v, int lane) {
  return {__shfl_sync(0xffffffffu, v.x, lane), __shfl_sync(0xffffffffu, v.e, lane)};
}
__device__ __forceinline__ Pair scan(Pair v, int lanes) {  // inclusive, over the first `lanes` lanes (a power of two)
  const int lane = threadIdx.x & 31;
  for (int d = 1; d < lanes; d <<= 1) {
    const Pair y = {__shfl_up_sync(0xffffffffu, v.x, d), __shfl_up_sync(0xffffffffu, v.e, d)};
    if (lane >= d) add(v, y);
  }
  return v;
}
__device__ __forceinline__ Pair over_warp(Pair v) {  // the warp's sum, in every lane
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) add(v, {__shfl_xor_sync(0xffffffffu, v.x, d), __shfl_xor_sync(0xffffffffu, v.e, d)});
  // (the lanes' additions differ in their order, and so may the last bits)
  return {__shfl_sync(0xffffffffu, v.x, 0), __shfl_sync(0xffffffffu, v.e, 0)};
}
// Two pairs side by side.
struct Pair2 {
  uint64_t x, e;
};
__device__ __forceinline__ Pair2 two_sum(uint64_t a, uint64_t b) {
  const uint64_t s = f2_add(a, b), bb = f2_sub(s, a);
  return {s, f2_add(f2_sub(a, f2_sub(s, bb)), f2_sub(b, bb))};
}
__device__ __forceinline__ Pair2 two_difference(uint64_t a, uint64_t b) {  // a - b
  const uint64_t s = f2_sub(a, b), bb = f2_sub(s, a);
  return {s, f2_sub(f2_sub(a, f2_sub(s, bb)), f2_add(b, bb))};
}
__device__ __forceinline__ void add(Pair2 &sum, Pair2 v) {
  const Pair2 s = two_sum(sum.x, v.x);
  sum.x = s.x;
  sum.e = f2_add(sum.e, f2_add(s.e, v.e));
}
__device__ __forceinline__ void add(Pair2 &sum, uint64_t v) {
  const Pair2 s = two_sum(sum.x, v);
  sum.x = s.x;
  sum.e = f2_add(sum.e, s.e);
}
__device__ __forceinline__ void split(Pair2 v, Pair &lo, Pair &hi) {
  f2_split(v.x, lo.x, hi.x);
  f2_split(v.e, lo.e, hi.e);
}
__device__ __forceinline__ void add(Pair &sum, float v) {
  const Pair s = two_sum(sum.x, v);
  sum.x = s.x;
  sum.e = __fadd_rn(sum.e, s.e);
}
// max(p - A q, 0), A a pair; the product's rounding is what an FMA gives back.
__device__ __forceinline__ Pair residual(float p, float q, Pair A) {
  const float m = __fmul_rn(q, A.x), lost = __fmaf_rn(q, A.e, __fmaf_rn(q, A.x, -m));
  Pair d = two_sum(p, -m);
  d.e = __fadd_rn(d.e, -lost);
  if (!positive(d)) d.x = d.e = 0.f;
  return d;
}
// (a p that is no probability gives no residual: it is not above 0, or its error is no number)
__device__ __forceinline__ Pair2 residual(uint64_t p, uint64_t q, Pair A) {
  Pair lo, hi;
  if (A.x == 1.f && A.e == 0.f) {  // after one refusal: the difference's sign is its value's, and its error's when that is 0
    split(two_difference(p, q), lo, hi);
    const bool l = lo.x > 0.f && lo.x < INFINITY, h = hi.x > 0.f && hi.x < INFINITY;
    return {f2(l ? lo.x : 0.f, h ? hi.x : 0.f), f2(l ? lo.e : 0.f, h ? hi.e : 0.f)};
  }
  const uint64_t ax = f2(A.x, A.x), m = f2_mul(q, ax);
  Pair2 d = two_difference(p, m);
  d.e = f2_sub(d.e, f2_fma(q, f2(A.e, A.e), f2_fma(q, ax, f2_sub(0ull, m))));
  split(d, lo, hi);
  float l, h;
  f2_split(f2_add(d.x, d.e), l, h);
  return {f2(l > 0.f ? lo.x : 0.f, h > 0.f ? hi.x : 0.f), f2(l > 0.f ? lo.e : 0.f, h > 0.f ? hi.e : 0.f)};
}
// 16 bytes of a row as probabilities, two by two.
template <typename E, bool ALL>
__device__ __forceinline__ void unpack(uint4 w, uint64_t (&x)[8 / sizeof(E)]) {
  const E *e = reinterpret_cast<const E *>(&w);
#pragma unroll
  for (int j = 0; j < 8 / (int)sizeof(E); ++j) {
    const float a = as_f32(e[2 * j]), b = as_f32(e[2 * j + 1]);
    x[j] = ALL ? f2(a, b) : f2(some(a), some(b));
  }
}

template <typename E, bool DRAFT>
__global__ void __launch_bounds__(kThreads, 2) tree_verify_kernel(const TreeVerifyArgs a) {
  constexpr int VEC = Row<E>::VEC;
  extern __shared__ __align__(16) uint8_t raw[];
  Shared &s = *reinterpret_cast<Shared *>(raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_rank(), ctas = cluster_size();
  const int req = blockIdx.x / ctas;
  cluster_arrive();  // (every CTA has begun before its shared memory is written from another)
  pdl_wait();
  pdl_trigger();
  if (rank == 0) {
    const Rows r = rows_of(a.cu_q, req, a.T, tid == 0 ? a.err : nullptr);
    const float u_last = a.u_last[req];
    const int row0 = a.rows ? a.rows[req] : r.first;
    int nodes = r.count;
    if (row0 < 0) {
      nodes = -1;  // not verified
    } else if (nodes > FM_MAX_NODES || (int64_t)row0 + nodes > a.R) {
      if (tid == 0) report(a.err, kDevErrLength, (unsigned)req, (unsigned)row0, (unsigned)row0 + (unsigned)nodes, 0u);
      nodes = 0;
    }
    cluster_wait();
    if (tid < (int)ctas) {
      put_remote(in_cta(smem_at(&s.first), tid), (uint32_t)row0);
      put_remote(in_cta(smem_at(&s.nodes), tid), (uint32_t)nodes);
      put_remote(in_cta(smem_at(&s.u_last), tid), __float_as_uint(fminf(fmaxf(u_last, 0.f), 1.f)));
    }
    for (int t = tid; t < nodes; t += kThreads) {
      const int row = r.first + t;
      int parent = a.parent[row], token = a.tokens[row];
      const float u = a.u[row];
      float p = 0.f, q = 0.f;
      if (t > 0 && (token < 0 || token >= a.V)) {
        report(a.err, kDevErrToken, (unsigned)req, (unsigned)t, (unsigned)token, 0u);
        token = -1;
      }
      if (parent < 0 || parent >= t) parent = -1;  // never reached: a child comes behind its parent
      if (parent >= 0 && token >= 0) {
        p = some(as_f32(reinterpret_cast<const E *>(a.p)[(int64_t)(row0 + parent) * a.sp + token]));
        if (DRAFT) q = some(as_f32(reinterpret_cast<const E *>(a.q)[(int64_t)(row0 + parent) * a.sq + token]));
      }
      for (uint32_t c = 0; c < ctas; ++c) {
        put_remote(in_cta(smem_at(&s.parent[t]), c), (uint32_t)parent);
        put_remote(in_cta(smem_at(&s.token[t]), c), (uint32_t)token);
        put_remote(in_cta(smem_at(&s.u[t]), c), __float_as_uint(u));
        put_remote(in_cta(smem_at(&s.p[t]), c), __float_as_uint(p));
        put_remote(in_cta(smem_at(&s.q[t]), c), __float_as_uint(q));
      }
    }
  } else {
    cluster_wait();
  }
  cluster_arrive();
  cluster_wait();
  // (from here on what decides the way is the same in every CTA: they meet equally often)
  const int first = s.first, nodes = s.nodes;
  int32_t *path = a.path + (int64_t)req * a.max_path;
  if (nodes <= 0) {
    if (rank == 0) {
      for (int64_t j = tid; j < a.max_path; j += kThreads) path[j] = -1;
      if (tid == 0) a.kept[req] = nodes, a.next[req] = -1;
    }
    return;
  }
  // What is left of the elements of block b of the row after node cur.
  auto left = [&](uint4 pw, uint4 qw, Pair A, int n_refused, int b, int shift, Pair2 (&x)[VEC / 2]) {
    uint64_t p2[VEC / 2];
    if (DRAFT && A.x > 0.f) {
      uint64_t q2[VEC / 2];
      unpack<E, true>(pw, p2);
      unpack<E, false>(qw, q2);
#pragma unroll
      for (int j = 0; j < VEC / 2; ++j) x[j] = residual(p2[j], q2[j], A);
      return;
    }
    unpack<E, false>(pw, p2);
#pragma unroll
    for (int j = 0; j < VEC / 2; ++j) x[j] = {p2[j], 0ull};
    if (!DRAFT && n_refused > 0) {
      uint32_t gone = 0u;  // elements of the block
#pragma unroll 1
      for (int i = 0; i < n_refused; ++i) {
        const int at = s.refused[i] + shift - b * VEC;
        if (at >= 0 && at < VEC) gone |= 1u << at;
      }
#pragma unroll
      for (int j = 0; j < VEC / 2; ++j)
        x[j].x &= ((gone >> (2 * j)) & 1u ? 0ull : 0xffffffffull) | ((gone >> (2 * j + 1)) & 1u ? 0ull : 0xffffffff00000000ull);
    }
  };
  // The warp's sum of what is left of the blocks [w0, w1).
  auto sum_blocks = [&](const Row<E> &p, const Row<E> &q, Pair A, int n_refused, int w0, int w1) -> Pair {
    constexpr int U = DRAFT ? 2 : 4;  // blocks under way at a time
    if (!DRAFT) {
      bool here = false;  // a refused token lies in them
      for (int i = lane; i < n_refused; i += 32) {
        const int at = (s.refused[i] + p.shift) / VEC;
        here |= at >= w0 && at < w1;
      }
      if (!__any_sync(0xffffffffu, here)) n_refused = 0;
    }
    Pair2 sum = {0ull, 0ull};
    for (int b0 = w0 + lane; b0 - lane < w1; b0 += 32 * U) {
      uint4 pw[U], qw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int b = b0 + 32 * u;
        pw[u] = qw[u] = make_uint4(0u, 0u, 0u, 0u);
        if (b < w1) {
          pw[u] = p.load(b);
          if (DRAFT && A.x > 0.f) qw[u] = q.load(b);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u == 0 || b0 - lane + 32 * u < w1) {
          Pair2 x[VEC / 2];
          left(pw[u], qw[u], A, n_refused, b0 + 32 * u, p.shift, x);
#pragma unroll
          for (int j = 0; j < VEC / 2; ++j) {
            if (DRAFT) add(sum, x[j]);
            else add(sum, x[j].x);
          }
        }
      }
    }
    Pair lo, hi;
    split(sum, lo, hi);
    add(lo, hi);
    return over_warp(lo);
  };
  // Where part `i` of 2^k even ones of the blocks [b0, b1) begins.
  auto part = [](int b0, int b1, int i, int k) -> int { return b0 + (int)((int64_t)(b1 - b0) * i >> k); };
  constexpr int kLogWarps = 4;
  static_assert(1 << kLogWarps == kWarps, "");
  const int log_parts = kLogWarps + 31 - __clz((int)ctas);  // (the cluster's size is a power of two)

  // The first warp's walk.
  int cur = 0, kept = 1, n_refused = 0, passes = 0, t = 0, part0 = 0, part1 = 0;
  Pair A = {0.f, 0.f}, S = {1.f, 0.f}, border = {0.f, 0.f}, before = {0.f, 0.f};
  bool summed = false;  // S and the warps' sums are those of (cur, A)
  bool ended = false;   // no child is left to try
  if (rank == 0 && tid == 0) path[0] = 0;

  // Goes on with the walk until a sum is wanted; the next order to the CTA's warps.
  auto walk = [&]() -> int {
    while (!ended) {
      int child = -1;  // the next child of cur behind node t
      if (kept < a.max_path)
        for (int b = (t + 1) & ~31; b < nodes; b += 32) {
          const int i = b + lane;
          const unsigned m = __ballot_sync(0xffffffffu, i > t && i < nodes && s.parent[i] == cur && s.token[i] >= 0);
          if (m) {
            child = b + __ffs(m) - 1;
            break;
          }
        }
      if (child < 0) {
        ended = true;
        break;
      }
      t = child;
      const float u = fminf(fmaxf(s.u[t], 0.f), 1.f);
      float p = s.p[t], q = s.q[t];
      const int token = s.token[t];
      bool take;
      if (DRAFT) {
        // (both sides scale with p and q, whose products would lose bits below 2^-126)
        if (fmaxf(p, q) < 1.f) p *= 0x1p64f, q *= 0x1p64f;
        const float m = __fmul_rn(u, q), lost = __fmaf_rn(u, q, -m);
        Pair wanted = times(S, m);
        wanted.e = __fmaf_rn(S.x, lost, wanted.e);
        take = less(wanted, residual(p, q, A));
      } else {
        bool gone = false;
        for (int i = lane; i < n_refused; i += 32) gone |= s.refused[i] == token;
        if (__any_sync(0xffffffffu, gone)) p = 0.f;
        take = less(times(S, u), {p, 0.f});
      }
      if (take) {
        if (rank == 0 && lane == 0) path[kept] = t;
        cur = t;
        ++kept;
        A = {0.f, 0.f};
        S = {1.f, 0.f};
        n_refused = 0;
        summed = false;
      } else if (DRAFT) {
        add(A, S);
        A = two_sum(A.x, A.e);
        return kSum;
      } else {
        add(S, -p);
        if (!positive(S)) S = {0.f, 0.f};
        if (lane == 0) s.refused[n_refused] = token;
        ++n_refused;
        __syncwarp();
      }
    }
    return summed ? kFind : kSum;
  };
  // The sums of all CTAs' warps, a power of two of them a lane.
  const int log_each = max(log_parts - 5, 0), each = 1 << log_each;
  auto part_sum = [&](int i) -> Pair { return i < 1 << log_parts ? s.part[(passes - 1) & 1][i] : Pair{0.f, 0.f}; };
  unsigned nonzero = 0u;  // lanes whose parts hold anything
  // After a sum: its value.
  auto after_sum = [&]() {
    Pair mine = part_sum(lane << log_each);
    for (int j = 1; j < each; ++j) add(mine, part_sum((lane << log_each) + j));
    nonzero = __ballot_sync(0xffffffffu, positive(mine));
    const Pair inc = scan(mine, 32);
    s.upto[lane] = inc;
    S = shuffle(inc, 31);
    S = two_sum(S.x, S.e);
    summed = S.x > 0.f;
    if (!summed && (!ended || n_refused > 0)) {  // nothing is left: the target's row as it was
      A = {0.f, 0.f};
      S = {1.f, 0.f};
      n_refused = 0;
    } else if (!summed) {  // the row itself is empty
      S = {0.f, 0.f};
    }
    __syncwarp();
  };
  // The part of the row that holds the border, and in `before` the sum of the parts before it.
  auto part_of_border = [&]() -> int {
    const unsigned past = __ballot_sync(0xffffffffu, less(border, s.upto[lane])) & nonzero;
    const int at = past ? __ffs(past) - 1 : 31 - __clz(nonzero | 1u);
    Pair upto = at > 0 ? s.upto[at - 1] : Pair{0.f, 0.f};
    int found = at << log_each;
    for (int j = 0; j < each; ++j) {
      const Pair v = part_sum((at << log_each) + j);
      if (!positive(v)) continue;
      found = (at << log_each) + j;
      before = upto;
      add(upto, v);
      if (less(border, upto)) break;
    }
    return found;
  };
  // The lane (of the first `n`) whose value takes the sum past the border, else the last with one above 0; `before`
  // becomes the sum of the lanes before it.  -1: every value is 0.
  auto past_border = [&](Pair v, int n) -> int {
    if (lane >= n) v = {0.f, 0.f};
    const bool some_left = positive(v);
    const unsigned any = __ballot_sync(0xffffffffu, some_left);
    const Pair inc = scan(v, kWarps);  // (n is at most that)
    Pair upto = before;
    add(upto, inc);
    const unsigned past = __ballot_sync(0xffffffffu, some_left && less(border, upto));
    if (!any) return -1;
    const int at = past ? __ffs(past) - 1 : 31 - __clz(any);
    upto = shuffle(inc, max(at - 1, 0));
    if (at > 0) add(before, upto);
    return at;
  };

  for (;;) {
    if (warp == 0) {
      int what = passes == 0 || !ended ? walk() : (summed ? kFind : kSum);
      if (ended && passes > 0 && !(S.x > 0.f)) what = kDone;
      if (what == kFind) {
        border = times(S, s.u_last);
        const int w = part_of_border();
        if (w / kWarps != (int)rank) {
          what = kDone;
        } else {
          const Row<E> p(a.p, a.sp, first + cur, (int)a.V);
          part0 = part(0, p.blocks(), w, log_parts);
          part1 = part(0, p.blocks(), w + 1, log_parts);
        }
      }
      if (lane == 0) {
        s.what = what;
        s.cur = cur;
        s.n_refused = n_refused;
        s.part0 = part0;
        s.part1 = part1;
        s.A = A;
      }
    }
    __syncthreads();
    const int what = s.what;
    if (what == kDone) break;
    // (a short part is taken block by block at once)
    const bool at_once = what == kFind && s.part1 - s.part0 <= 64;
    const int row = first + s.cur, refused = s.n_refused;
    const Pair A2 = s.A;
    const Row<E> p(a.p, a.sp, row, (int)a.V), q(DRAFT ? a.q : a.p, DRAFT ? a.sq : a.sp, row, (int)a.V, p.shift);
    const int b0 = what == kSum ? 0 : s.part0, b1 = what == kSum ? p.blocks() : s.part1;
    const int i = what == kSum ? (int)rank * kWarps + warp : warp, k = what == kSum ? log_parts : kLogWarps;
    Pair sum = {0.f, 0.f};
    if (!at_once) sum = sum_blocks(p, q, A2, refused, part(b0, b1, i, k), part(b0, b1, i + 1, k));
    if (what == kSum) {
      if (lane < (int)ctas) {
        Pair *to = &s.part[passes & 1][i];
        put_remote(in_cta(smem_at(&to->x), lane), __float_as_uint(sum.x));
        put_remote(in_cta(smem_at(&to->e), lane), __float_as_uint(sum.e));
      }
      cluster_arrive();
      cluster_wait();
      ++passes;
      if (warp == 0) after_sum();
      continue;
    }
    if (lane == 0) s.warp[warp] = sum;
    __syncthreads();
    // The border lies in a sixteenth of the part: the first warp takes it block by block.
    if (warp == 0) {
      int w0 = b0, w1 = b1;
      if (!at_once) {
        const int w = max(past_border(s.warp[lane & (kWarps - 1)], kWarps), 0);
        w0 = part(b0, b1, w, kLogWarps);
        w1 = part(b0, b1, w + 1, kLogWarps);
      }
      int last = -1;  // the last token so far of which anything is left
      for (int c0 = w0; c0 < w1; c0 += 32) {
        const int b = c0 + lane;
        uint4 pw = make_uint4(0u, 0u, 0u, 0u), qw = pw;
        if (b < w1) {
          pw = p.load(b);
          if (DRAFT && A2.x > 0.f) qw = q.load(b);
        }
        Pair2 x2[VEC / 2];
        Pair x[VEC], sum = {0.f, 0.f};
        left(pw, qw, A2, refused, b, p.shift, x2);
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) split(x2[j], x[2 * j], x[2 * j + 1]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) add(sum, x[j]);
        const Pair inc = scan(sum, 32);
        Pair run = before;
        add(run, inc);
        const bool some_left = positive(sum);
        const unsigned any = __ballot_sync(0xffffffffu, some_left);
        const unsigned past = __ballot_sync(0xffffffffu, some_left && less(border, run));
        if (any) {
          const int from = past ? __ffs(past) - 1 : 31 - __clz(any);
          // in that lane: the first token past the border, else the last with anything left
          const Pair prior = shuffle(inc, max(from - 1, 0));
          run = before;
          if (from > 0) add(run, prior);
          int pick = -1;
          bool done = false;
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            add(run, x[j]);
            if (positive(x[j]) && !done) {
              pick = b * VEC - p.shift + j;
              done = less(border, run);
            }
          }
          last = __shfl_sync(0xffffffffu, pick, from);
          if (past) break;
        }
        add(before, shuffle(inc, 31));
      }
      if (lane == 0) a.next[req] = last;
    }
    break;
  }
  if (rank == 0 && warp == 0) {
    for (int j = kept + lane; j < a.max_path; j += 32) path[j] = -1;
    if (lane == 0) {
      a.kept[req] = kept;
      if (!(S.x > 0.f)) a.next[req] = -1;
    }
  }
}

template <typename E, bool DRAFT>
cudaError_t launch(const TreeVerifyArgs &a, unsigned ctas, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.n * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, tree_verify_kernel<E, DRAFT>, a);
}
static_assert(sizeof(Shared) <= 48 * 1024, "shared memory without an attribute");

}  // namespace

cudaError_t launch_tree_verify(const TreeVerifyArgs &a, cudaStream_t st) {
  // As many CTAs a request as run at once (two a SM; clusters of 4 and 8 leave some SMs out), with a thousand
  // tokens each at least.  Where trees branch (more nodes than a path has) and children were drawn, a request
  // sums its row once a refusal, and parts of 16,000 tokens are worth up to four CTAs a SM.  (max_path is all that
  // the host knows of the trees' shape: with more room in a path than a tree has nodes, trees of 8 are taken for
  // chains, 100 over 64,000 tokens 35.5 -> 39.2 us, 150 over 128,000 72 -> 87, 64 of bf16 31.3 -> 32.9.)  By CTAs a
  // request (us, L2 flushed; 8 nodes in trees of paths of 4 to 6, chains of 8):
  //   requests, tokens, rows of                          1     2     4     8
  //     1   128,000  bf16, target and draft           29.3  22.2  19.1  17.1
  //    64   128,000  bf16, both, trees                 111  66.2  45.8  41.6
  //    64   128,000  bf16, both, chains               45.7  31.4  29.3  37.5
  //    64    32,000  bf16, both, trees                37.5  27.3  25.2  31.4
  //   100    64,000  fp32, both, trees                86.7  55.9  41.6  49.8
  //   100    64,000  fp32, both, chains               33.4  27.3  35.5  41.6
  //   150   128,000  fp32, both, trees                 132  96.9  76.4  80.5
  //   150   128,000  fp32, both, chains               55.9  45.7  60.0  74.4
  //   200    32,000  fp32, both, trees                64.2  47.8  47.8  64.2
  //    48   100,003  bf16, target                     33.4  25.2  21.2  29.3
  //    76   100,000  fp32, target                     37.4  25.2  29.3  35.5
  //   150    64,000  bf16, target                     27.3  23.2  37.5  53.9
  //   230    64,000  bf16, target                     30.8  38.9  49.8  74.4
  //    16     4,000  fp32, both, trees                23.2  21.2  21.2  23.2
  const int64_t sms = current_device_sm_count();
  const bool many_sums = a.q && a.R > a.n * a.max_path;
  unsigned ctas = kMostCtas;
  for (; ctas > 1; ctas /= 2) {
    const int64_t most = many_sums && a.V / ctas >= 16000 ? 4 * sms : 2 * sms - (ctas >= 4 ? sms / 10 : 0);
    if (a.n * ctas <= most && a.V >= 1024 * (int64_t)ctas) break;
  }
  const bool draft = a.q != nullptr;
  if (a.dtype == FM_F32) return draft ? launch<float, true>(a, ctas, st) : launch<float, false>(a, ctas, st);
  if (a.dtype == FM_BF16) return draft ? launch<__nv_bfloat16, true>(a, ctas, st) : launch<__nv_bfloat16, false>(a, ctas, st);
  return draft ? launch<__half, true>(a, ctas, st) : launch<__half, false>(a, ctas, st);
}

}  // namespace fm
