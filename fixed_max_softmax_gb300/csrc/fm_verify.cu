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
// the p and q that their tests compare into every CTA's shared memory; from there all CTAs
// walk alike, and meet only to sum what is left over the vocabulary, once a refused child and
// once at the end: each sums an even part of the row, and the parts' sums go to every CTA's shared
// memory.  A walk without a refusal reads one row of the vocabulary in all.
// Sums are 64-bit, as are the tests: they are compared with a random number, and a sum that is off by
// 2^-24 would pick another token than the definition does at every border that the number falls next to.
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
__device__ __forceinline__ void put_remote(uint32_t addr, double v) {
  asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(addr), "d"(v) : "memory");
}

__device__ __forceinline__ float as_f32(float x) { return x; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float as_f32(__half x) { return __half2float(x); }
// A probability: what is negative, infinite or no number counts as 0.
__device__ __forceinline__ float some(float x) { return x > 0.f && x < INFINITY ? x : 0.f; }

struct Shared {
  int parent[FM_MAX_NODES], token[FM_MAX_NODES];  // token -1: outside the vocabulary
  float u[FM_MAX_NODES], p[FM_MAX_NODES], q[FM_MAX_NODES];
  int first, nodes;             // as the first CTA read them
  int refused[FM_MAX_NODES];    // tokens taken out of p (children that were chosen)
  double cta[2][kMostCtas];     // the CTAs' sums, of alternate passes
  double warp[kWarps];          // this CTA's warps' sums
};

// A row of one model in blocks of 16 bytes, block 0 beginning at the boundary before the row's start:
// element `e` of block b is element b * VEC - shift + e of the row.
template <typename E>
struct Row {
  static constexpr int VEC = 16 / (int)sizeof(E);
  const E *at;  // of block 0
  int64_t shift, V;

  __device__ __forceinline__ Row(const void *base, int64_t stride, int64_t row, int64_t V_) : V(V_) {
    const E *p = reinterpret_cast<const E *>(base) + row * stride;
    shift = (int64_t)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(E));
    at = p - shift;
  }
  __device__ __forceinline__ int64_t blocks() const { return (V + shift + VEC - 1) / VEC; }
  // block b as another row of alignment `s` has it
  __device__ __forceinline__ void load(int64_t b, int64_t s, float (&x)[VEC]) const {
    const int64_t i = b * VEC - s;  // in the row
    if (s == shift && i >= 0 && i + VEC <= V) {
      const uint4 w = *reinterpret_cast<const uint4 *>(at + b * VEC);
      const E *e = reinterpret_cast<const E *>(&w);
#pragma unroll
      for (int j = 0; j < VEC; ++j) x[j] = some(as_f32(e[j]));
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) x[j] = i + j >= 0 && i + j < V ? some(as_f32(at[shift + i + j])) : 0.f;
    }
  }
};

template <typename E, bool DRAFT>
__global__ void __launch_bounds__(kThreads) tree_verify_kernel(const TreeVerifyArgs a) {
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
    int nodes = r.count;
    if (nodes > FM_MAX_NODES) {
      if (tid == 0) report(a.err, kDevErrLength, (unsigned)req, (unsigned)r.first, (unsigned)(r.first + r.count), 0u);
      nodes = 0;
    }
    cluster_wait();
    if (tid < (int)ctas) {
      put_remote(in_cta(smem_at(&s.first), tid), (uint32_t)r.first);
      put_remote(in_cta(smem_at(&s.nodes), tid), (uint32_t)nodes);
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
        p = some(as_f32(reinterpret_cast<const E *>(a.p)[(int64_t)(r.first + parent) * a.sp + token]));
        if (DRAFT) q = some(as_f32(reinterpret_cast<const E *>(a.q)[(int64_t)(r.first + parent) * a.sq + token]));
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
  if (nodes == 0) {
    if (rank == 0) {
      for (int64_t j = tid; j < a.max_path; j += kThreads) path[j] = -1;
      if (tid == 0) a.kept[req] = 0, a.next[req] = -1;
    }
    return;
  }
  int cur = 0, kept = 1, n_refused = 0, passes = 0;
  double A = 0.0, S = 1.0;
  bool summed = false;  // S and the warps' sums are those of (cur, A)
  if (rank == 0 && tid == 0) path[0] = 0;

  // this warp's blocks of the row
  int64_t w0 = 0, w1 = 0;
  // What is left of block b of the row, given A and the refused tokens.
  auto left = [&](const Row<E> &p, const Row<E> &q, int64_t b, double (&x)[VEC]) {
    float f[VEC];
    p.load(b, p.shift, f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[j] = (double)f[j];
    if (DRAFT && A > 0.0) {
      q.load(b, p.shift, f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) x[j] = fmax(x[j] - A * (double)f[j], 0.0);
    }
    for (int i = 0; i < n_refused; ++i) {
      const int64_t at = (int64_t)s.refused[i] + p.shift - b * VEC;
      if (at >= 0 && at < VEC) {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (j == at) x[j] = 0.0;
      }
    }
  };
  // S = sum of what is left of row cur; every thread of the cluster.
  auto sum_up = [&]() {
    const Row<E> p(a.p, a.sp, first + cur, a.V), q(DRAFT ? a.q : a.p, DRAFT ? a.sq : a.sp, first + cur, a.V);
    const int64_t nb = p.blocks(), parts = (int64_t)ctas * kWarps, mine = (int64_t)rank * kWarps + warp;
    w0 = nb * mine / parts;
    w1 = nb * (mine + 1) / parts;
    double sum = 0.0;
    for (int64_t b = w0 + lane; b < w1; b += 32) {
      double x[VEC];
      left(p, q, b, x);
#pragma unroll
      for (int j = 0; j < VEC; ++j) sum += x[j];
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (lane == 0) s.warp[warp] = sum;
    __syncthreads();
    double *slot = s.cta[passes & 1];
    if (tid < (int)ctas) {
      double x = 0.0;
      for (int w = 0; w < kWarps; ++w) x += s.warp[w];
      put_remote(in_cta(smem_at(slot + rank), tid), x);
    }
    cluster_arrive();
    cluster_wait();
    S = 0.0;
    for (uint32_t c = 0; c < ctas; ++c) S += slot[c];
    ++passes;
  };

  int t = 0;
  while (kept < a.max_path) {
    // the next child of cur behind node t
    int child = -1;
    for (int b = (t + 1) & ~31; b < nodes; b += 32) {
      const int i = b + lane;
      const unsigned m = __ballot_sync(0xffffffffu, i > t && i < nodes && s.parent[i] == cur && s.token[i] >= 0);
      if (m) {
        child = b + __ffs(m) - 1;
        break;
      }
    }
    if (child < 0) break;
    t = child;
    const double u = (double)fminf(fmaxf(s.u[t], 0.f), 1.f), p = (double)s.p[t], q = (double)s.q[t];
    const int token = s.token[t];
    bool take;
    double rest = 0.0;
    if (DRAFT) {
      take = u * q * S < fmax(p - A * q, 0.0);
    } else {
      rest = p;
      for (int i = 0; i < n_refused; ++i)
        if (s.refused[i] == token) rest = 0.0;
      take = u * S < rest;
    }
    if (take) {
      if (rank == 0 && tid == 0) path[kept] = t;
      cur = t;
      ++kept;
      A = 0.0;
      S = 1.0;
      n_refused = 0;
      summed = false;
      __syncthreads();  // (the refused tokens have been read)
    } else if (DRAFT) {
      A += S;
      sum_up();
      summed = S > 0.0;
      if (!summed) A = 0.0, S = 1.0;  // nothing is left: the target's row as it was
    } else {
      S = fmax(S - rest, 0.0);
      __syncthreads();
      if (tid == 0) s.refused[n_refused] = token;
      ++n_refused;
      __syncthreads();
    }
  }
  if (!summed) {
    sum_up();
    if (!(S > 0.0) && n_refused > 0) {
      __syncthreads();
      n_refused = 0;
      sum_up();
    }
  }
  if (rank == 0) {
    for (int64_t j = kept + tid; j < a.max_path; j += kThreads) path[j] = -1;
    if (tid == 0) {
      a.kept[req] = kept;
      if (!(S > 0.0)) a.next[req] = -1;
    }
  }
  if (!(S > 0.0)) return;
  // the CTA, then the warp, whose part holds the border
  const float ul = a.u_last[req];
  const double border = (double)fminf(fmaxf(ul, 0.f), 1.f) * S;
  const double *slot = s.cta[(passes - 1) & 1];
  double upto = 0.0, before = 0.0;
  int owner = -1;
  bool found = false;
  for (int c = 0; c < (int)ctas && !found; ++c) {
    if (slot[c] > 0.0) owner = c, before = upto;
    upto += slot[c];
    found = upto > border;
  }
  if ((int)rank != owner) return;
  upto = before;
  found = false;
  owner = -1;
  for (int w = 0; w < kWarps && !found; ++w) {
    if (s.warp[w] > 0.0) owner = w, before = upto;
    upto += s.warp[w];
    found = upto > border;
  }
  if (warp != owner) return;
  const Row<E> p(a.p, a.sp, first + cur, a.V), q(DRAFT ? a.q : a.p, DRAFT ? a.sq : a.sp, first + cur, a.V);
  int64_t last = -1;  // the last token so far of which anything is left
  for (int64_t b0 = w0; b0 < w1; b0 += 32) {
    const int64_t b = b0 + lane;
    double x[VEC], sum = 0.0;
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[j] = 0.0;
    if (b < w1) left(p, q, b, x);
#pragma unroll
    for (int j = 0; j < VEC; ++j) sum += x[j];
    double inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += y;
    }
    const unsigned any = __ballot_sync(0xffffffffu, sum > 0.0);
    const unsigned past = __ballot_sync(0xffffffffu, sum > 0.0 && before + inc > border);
    if (any) {
      const int from = past ? __ffs(past) - 1 : 31 - __clz(any);
      // in that lane: the first token past the border, else the last with anything left
      double run = __shfl_up_sync(0xffffffffu, inc, 1);
      run = before + (lane > 0 ? run : 0.0);
      int64_t pick = -1;
      bool done = false;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        run += x[j];
        if (x[j] > 0.0 && !done) {
          pick = b * VEC - p.shift + j;
          done = run > border;
        }
      }
      last = __shfl_sync(0xffffffffu, pick, from);
      if (past) break;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (lane == 0) a.next[req] = (int32_t)last;
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
  // as many CTAs a request as two a SM allow, each with some thousand tokens at least
  unsigned ctas = kMostCtas;
  while (ctas > 1 && ((int64_t)a.n * ctas > 2 * current_device_sm_count() || a.V < 2048 * (int64_t)ctas)) ctas /= 2;
  const bool draft = a.q != nullptr;
  if (a.dtype == FM_F32) return draft ? launch<float, true>(a, ctas, st) : launch<float, false>(a, ctas, st);
  if (a.dtype == FM_BF16) return draft ? launch<__nv_bfloat16, true>(a, ctas, st) : launch<__nv_bfloat16, false>(a, ctas, st);
  return draft ? launch<__half, true>(a, ctas, st) : launch<__half, false>(a, ctas, st);
}

}  // namespace fm
