// fm_paged.cu -- the bookkeeping of a paged key/value cache, on the GPU.
//
// fm_paged_extend: with base_i = (request i released ? 0 : kv_i), P(x) = ceil(x / page_size)
//   pages given back  G = sum over released i of P(kv_i): pushed on the list of free pages in
//                     request order, then table order
//   pages taken       F = sum_i P(base_i + new_i) - P(base_i): popped off the list's top in the
//                     same order, page e of the call being free[count + G - 1 - e]
//   token t of request i at position p = base_i + t - cu_i:  slot = table[i][p / page_size] *
//                     page_size + p mod page_size
// One cluster of CTAs moves the pages: every CTA takes the prefix sums of all requests for itself
// (12 bytes a request, read through L2), so that the CTAs meet only once, between the last read of
// the old state and the first write of the new one, which is what allows kv_len, free_count and the
// rows of reused requests to be updated in place.  Where the slots have room for up to 4,096 tokens the
// same CTA fills them, a token's page taken from the free list by its rank; where for more, a second
// kernel over the whole GPU does, from the finished table (336,704 tokens of 96 requests: 29.8 us by the
// cluster alone, 11.1 by the two).  The room decides, not the tokens, whose number is on the device: all of it is
// filled, with -1 behind the last token.  Bound by the latency of a few dependent loads, then by 12 bytes a slot.
//
// fm_paged_write: a copy of rows to their slots, bound by HBM (each row read and written once): 53,013
// tokens of 8 heads, D = 128, in 72.5 us, 89 % of the copy rate.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <limits.h>

#include <atomic>
#include <type_traits>

#include "fm_internal.h"

namespace fm {
namespace {

constexpr int kExtThreads = 1024;
constexpr int kExtWarps = kExtThreads / 32;

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The request that element e belongs to: the last i with pre[i] <= e (pre[0] = 0, ascending;
// empty requests are passed over because their successor has the same start).
__device__ __forceinline__ int owner(const int32_t *pre, int n, int e) {
  int lo = 0, hi = n;  // pre[lo] <= e < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= e) lo = mid; else hi = mid;
  }
  return lo;
}

struct Sums {
  long long tok, give, take;
};
__device__ __forceinline__ Sums add(const Sums &a, const Sums &b) {
  return Sums{a.tok + b.tok, a.give + b.give, a.take + b.take};
}
__device__ __forceinline__ Sums shfl_up(const Sums &a, int d) {
  return Sums{__shfl_up_sync(0xffffffffu, a.tok, d), __shfl_up_sync(0xffffffffu, a.give, d),
              __shfl_up_sync(0xffffffffu, a.take, d)};
}

__device__ __forceinline__ int pages_of(int x, int ps) { return (int)(((unsigned)x + (unsigned)ps - 1u) / (unsigned)ps); }

// Slots and positions of the T tokens (-1 from there to max_tokens), four to a thread: one search,
// and most often one page.  request_of(token), start(request), base(request): a request's first
// token and what it held before, page(request, j): its j-th page.
template <typename R, typename S, typename B, typename P>
__device__ __forceinline__ void put_tokens(const PagedExtendArgs &a, int T, int first, int step, R request_of, S start, B base,
                                           P page) {
  const long long cap = a.max_tokens;
  const int ps = (int)a.page_size;
  for (long long q = first; q * 4 < cap; q += step) {
    const long long t0 = q * 4;
    long long slot[4];
    int pos[4];
    int i = t0 < T ? request_of((int)t0) : 0;
    int last_i = -1, end = 0, shift = 0, last_page = -1, pg = 0;  // shift: position of the request's token 0 of this call
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const long long t = t0 + u;
      slot[u] = -1;
      pos[u] = -1;
      if (t < T) {
        if (last_i < 0 || t >= end) {
          while (t >= start(i + 1)) ++i;
          end = start(i + 1);
          shift = base(i) - start(i);
          last_page = -1;
          last_i = i;
        }
        const int p = (int)t + shift;
        const int j = p / ps;
        if (j != last_page) {
          pg = page(i, j);
          last_page = j;
        }
        pos[u] = p;
        slot[u] = (long long)pg * ps + (p - j * ps);
      }
    }
    if (t0 + 4 <= cap && ((reinterpret_cast<uintptr_t>(a.slots) | reinterpret_cast<uintptr_t>(a.positions)) & 15) == 0) {
      *reinterpret_cast<longlong2 *>(a.slots + t0) = make_longlong2(slot[0], slot[1]);
      *reinterpret_cast<longlong2 *>(a.slots + t0 + 2) = make_longlong2(slot[2], slot[3]);
      *reinterpret_cast<int4 *>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
      for (int u = 0; u < 4 && t0 + u < cap; ++u) {
        a.slots[t0 + u] = slot[u];
        a.positions[t0 + u] = pos[u];
      }
    }
  }
}

__global__ void __launch_bounds__(kExtThreads) paged_extend_kernel(const PagedExtendArgs a) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ int32_t smem[];
  const int n = (int)a.n, ps = (int)a.page_size;
  int32_t *tok_pre = smem;             // [n + 1] exclusive prefix sums of the new tokens
  int32_t *give_pre = smem + (n + 1);  // ... of the pages given back
  int32_t *take_pre = smem + 2 * (n + 1);  // ... of the pages taken
  int32_t *base = smem + 3 * (n + 1);  // [n]
  __shared__ Sums warp_sum[kExtWarps], carry_s;
  __shared__ int bad_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x, nctas = gridDim.x;  // the grid is one cluster
  if (tid == 0) {
    carry_s = Sums{0, 0, 0};
    bad_s = 0;
  }
  const int count = a.free_count[0];
  bool bad = count < 0 || count > a.num_pages;
  __syncthreads();
  for (int c0 = 0; c0 < n; c0 += kExtThreads) {
    const int i = c0 + tid;
    Sums v = {0, 0, 0};
    int b = 0;
    if (i < n) {
      const int nw = a.new_len[i], kv = a.kv_len[i];
      const bool rel = a.release && a.release[i] != 0;
      b = rel ? 0 : kv;
      // a length that cannot be, or a table row too short for it: the call changes nothing
      if (nw < 0 || kv < 0 || (long long)b + nw > INT_MAX - ps || kv > INT_MAX - ps ||
          pages_of(kv, ps) > a.table_width || pages_of(b + nw, ps) > a.table_width) {
        bad = true;
        b = 0;
      } else {
        v.tok = nw;
        v.give = rel ? pages_of(kv, ps) : 0;
        v.take = pages_of(b + nw, ps) - pages_of(b, ps);
      }
    }
    Sums inc = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Sums u = shfl_up(inc, d);
      if (lane >= d) inc = add(inc, u);
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    if (warp == 0) {
      Sums w = warp_sum[lane];
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const Sums u = shfl_up(w, d);
        if (lane >= d) w = add(w, u);
      }
      warp_sum[lane] = w;
    }
    __syncthreads();
    const Sums carry = carry_s;
    Sums ex = add(carry, inc);
    if (warp > 0) ex = add(ex, warp_sum[warp - 1]);
    if (i < n) {
      // sums past 2^31 are refused below; what is stored for them is never used
      tok_pre[i] = (int)(ex.tok - v.tok);
      give_pre[i] = (int)(ex.give - v.give);
      take_pre[i] = (int)(ex.take - v.take);
      base[i] = b;
    }
    __syncthreads();
    if (tid == 0) carry_s = add(carry, warp_sum[kExtWarps - 1]);
    __syncthreads();
  }
  if (bad) bad_s = 1;
  __syncthreads();
  const Sums total = carry_s;
  if (tid == 0) {
    tok_pre[n] = (int)total.tok;
    give_pre[n] = (int)total.give;
    take_pre[n] = (int)total.take;
  }
  int status = 0;
  if (bad_s || total.tok > a.max_tokens || count + total.give > a.num_pages) status = -1;
  else if (total.take > count + total.give) status = (int)(total.take - count - total.give);
  const bool ok = status == 0;
  __syncthreads();
  const int T = ok ? (int)total.tok : 0, back = ok ? (int)total.give : 0, fresh = ok ? (int)total.take : 0;
  const int g0 = rank * kExtThreads + tid, gstep = nctas * kExtThreads;
  for (int e = g0; e < back; e += gstep) {
    const int i = owner(give_pre, n, e);
    a.free_pages[count + e] = a.table[i * a.table_stride + (e - give_pre[i])];
  }
  // every CTA has read the old lengths, count and table rows, and the pushed pages are visible
  cluster_sync();
  const int top = count + back;
  for (int e = g0; e < fresh; e += gstep) {
    const int i = owner(take_pre, n, e);
    a.table[i * a.table_stride + pages_of(base[i], ps) + (e - take_pre[i])] = a.free_pages[top - 1 - e];
  }
  for (int i = g0; i <= n; i += gstep) {
    a.cu_q[i] = ok ? tok_pre[i] : 0;
    if (i < n && ok) a.kv_out[i] = base[i] + (tok_pre[i + 1] - tok_pre[i]);
    // a refused call leaves the lengths as they were
    else if (i < n && a.kv_out != a.kv_len) a.kv_out[i] = a.kv_len[i];
  }
  if (rank == 0 && tid == 0) {
    *a.free_out = top - fresh;
    *a.status = status;
  }
  if (a.slots_apart) return;
  put_tokens(a, T, g0, gstep, [&](int x) { return owner(tok_pre, n, x); }, [&](int i) { return tok_pre[i]; },
             [&](int i) { return base[i]; },
             [&](int i, int j) {
               const int have = pages_of(base[i], ps);
               return j < have ? a.table[i * a.table_stride + j] : a.free_pages[top - 1 - (take_pre[i] + j - have)];
             });
}

// Slots and positions of many tokens, after the kernel above: its cu_q and lengths say which request
// and position a token is, its table the page.
__global__ void __launch_bounds__(256) paged_slots_kernel(const PagedExtendArgs a) {
  pdl_wait();
  pdl_trigger();
  const int n = (int)a.n;
  const int32_t *cu = a.cu_q;
  put_tokens(a, cu[n], blockIdx.x * 256 + threadIdx.x, gridDim.x * 256, [&](int x) { return owner(cu, n, x); },
             [&](int i) { return cu[i]; }, [&](int i) { return a.kv_out[i] - (cu[i + 1] - cu[i]); },
             [&](int i, int j) { return a.table[i * a.table_stride + j]; });
}

// ---------------------------------------------------------------- cache writes
struct WriteArgs {
  View k, v, kc, vc;
  const int64_t *slots;
  unsigned int *err;
  int ps_shift;  // log2(page size), -1: not a power of two
};

// One row piece of `VEC` elements (16 bytes, or one element where layout or alignment ask for
// it) of K and of V a thread and step, two steps in flight.
template <typename E, int VEC>
__global__ void __launch_bounds__(256) paged_write_kernel(const WriteArgs a) {
  pdl_wait();
  pdl_trigger();
  using V = typename std::conditional<sizeof(E) * VEC == 16, uint4, E>::type;
  const unsigned per_head = (unsigned)(a.k.D / VEC), per_tok = per_head * (unsigned)a.k.H;
  const int64_t total = a.k.S * (int64_t)per_tok;
  const int64_t ps = a.kc.S, n_slots = a.kc.B * ps;
  const int64_t step = (int64_t)gridDim.x * 256;
  auto at = [](const View &x, int64_t b, int64_t h, int64_t s, int64_t d) -> E * {
    return reinterpret_cast<E *>(const_cast<void *>(x.ptr)) + b * x.sB + h * x.sH + s * x.sS + d * x.sD;
  };
  for (int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x; i0 < total; i0 += 2 * step) {
    V kx[2], vx[2];
    int64_t slot[2], dst_b[2], dst_s[2];
    unsigned h[2], d[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int64_t i = i0 + u * step;
      slot[u] = -1;
      if (i >= total) continue;
      const int64_t t = total <= UINT_MAX ? (int64_t)((unsigned)i / per_tok) : i / per_tok;
      const unsigned c = (unsigned)(i - t * per_tok);
      h[u] = c / per_head;
      d[u] = (c - h[u] * per_head) * VEC;
      slot[u] = a.slots[t];
      if (slot[u] >= n_slots) {  // never written: reported by fm_sync_status
        if (a.err && atomicCAS(a.err, 0u, (unsigned)kDevErrSlot) == 0u) {
          a.err[1] = (unsigned)t;
          a.err[2] = (unsigned)(slot[u] & 0xffffffffll);
          a.err[3] = (unsigned)(slot[u] >> 32);
        }
        slot[u] = -1;
      }
      if (slot[u] < 0) continue;
      dst_b[u] = a.ps_shift >= 0 ? slot[u] >> a.ps_shift : slot[u] / ps;
      dst_s[u] = slot[u] - dst_b[u] * ps;
      kx[u] = *reinterpret_cast<const V *>(at(a.k, 0, h[u], t, d[u]));
      vx[u] = *reinterpret_cast<const V *>(at(a.v, 0, h[u], t, d[u]));
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (slot[u] < 0) continue;
      *reinterpret_cast<V *>(at(a.kc, dst_b[u], h[u], dst_s[u], d[u])) = kx[u];
      *reinterpret_cast<V *>(at(a.vc, dst_b[u], h[u], dst_s[u], d[u])) = vx[u];
    }
  }
}

bool rows16(const View &x, int64_t es) {
  auto ok = [&](int64_t s, int64_t n) { return n <= 1 || (s * es) % 16 == 0; };
  return x.sD == 1 && reinterpret_cast<uintptr_t>(x.ptr) % 16 == 0 && ok(x.sS, x.S) && ok(x.sH, x.H) && ok(x.sB, x.B);
}

}  // namespace

cudaError_t launch_paged_extend(const PagedExtendArgs &args, cudaStream_t st) {
  PagedExtendArgs a = args;
  const size_t smem = (size_t)(4 * (a.n + 1)) * 4;
  static std::atomic<bool> attr_set[64] = {};  // once per device, so never while a stream is captured after a first call
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !attr_set[dev]) {
    e = cudaFuncSetAttribute(paged_extend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * (kMaxSeqs + 1) * 4);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) attr_set[dev] = true;
  }
  // one CTA for up to 4,096 tokens (one pass of its threads); beyond that a cluster of 8 for the
  // pages and a kernel of its own for the tokens
  a.slots_apart = a.max_tokens > 4096 ? 1 : 0;
  const unsigned ctas = a.slots_apart ? 8 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kExtThreads);
  cfg.dynamicSmemBytes = smem;
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
  e = cudaLaunchKernelEx(&cfg, paged_extend_kernel, a);
  if (e != cudaSuccess || !a.slots_apart) return e;
  const int64_t want = (a.max_tokens + 1023) / 1024, cap = (int64_t)current_device_sm_count() * 8;
  return launch_pdl(paged_slots_kernel, dim3((unsigned)(want < cap ? want : cap)), dim3(256), 0, st, a);
}

cudaError_t launch_paged_write(const View &k, const View &v, const int64_t *slots, const View &kc, const View &vc,
                               unsigned int *err, cudaStream_t st) {
  WriteArgs a;
  a.k = k;
  a.v = v;
  a.kc = kc;
  a.vc = vc;
  a.slots = slots;
  a.err = err;
  a.ps_shift = -1;
  for (int s = 0; s < 31; ++s)
    if (((int64_t)1 << s) == kc.S) a.ps_shift = s;
  const int64_t es = k.dtype == FM_F32 ? 4 : 2;
  const bool vec = rows16(k, es) && rows16(v, es) && rows16(kc, es) && rows16(vc, es);
  const int64_t total = k.S * k.H * (vec ? k.D * es / 16 : k.D);
  if (total == 0) return cudaSuccess;
  const int64_t want = (total + 511) / 512, cap = (int64_t)current_device_sm_count() * 16;
  const dim3 grid((unsigned)(want < cap ? want : cap));
  if (es == 4)
    return vec ? launch_pdl(paged_write_kernel<float, 4>, grid, dim3(256), 0, st, a)
               : launch_pdl(paged_write_kernel<float, 1>, grid, dim3(256), 0, st, a);
  return vec ? launch_pdl(paged_write_kernel<uint16_t, 8>, grid, dim3(256), 0, st, a)
             : launch_pdl(paged_write_kernel<uint16_t, 1>, grid, dim3(256), 0, st, a);
}

}  // namespace fm
