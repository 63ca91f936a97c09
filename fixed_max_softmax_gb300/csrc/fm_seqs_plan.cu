// fm_seqs_plan.cu -- the work list of one attention call over requests of different lengths, and
// the merge of units that were cut along their keys.
//
// Lengths live on the device, so the list is made there: one CTA reads them, decides how far
// to cut, and writes one entry per piece of work; the attention kernel's CTAs take entries in
// order from a counter.  Order: request, key head, range of keys, and the unit of queries
// running fastest (longest first), so that the CTAs at work at one moment mostly read the same
// key tiles, from L2.  A unit is cut into equal ranges of keys when it holds more than 2 / 3 of
// an even share of the work (512-token chunks over 32k keys: 404 us; cut at a whole share 518, at a
// third 425), and long pieces then go first, so that no CTA is left with one at the
// end (440 -> 413 us when that came); a cut unit's pieces leave unnormalised sums (o, max, sum) that
// seqs_merge_kernel joins in key order, so the result does not depend on which CTA did what.  The
// plan takes 8 to 16 us (one CTA, a few dependent passes), the merge 3 to 8.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "fm_seqs.cuh"

namespace fm {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kMergeRows = 8;  // warps of a merge CTA

struct PlanArgs {
  SeqsLens lens;
  int64_t n;
  int Hk, causal, window;
  SeqsGeom g;
  unsigned int *counters;
  int4 *req;  // per request: {first query row, queries, keys, first key row}, {units, tiles a piece, pieces, slot base}
  SeqsItem *items;
  SeqsMerge *merges;
  unsigned int *err;
};

// Exclusive prefix sum of v over the CTA in thread order; `total` gets the sum.
__device__ __forceinline__ long long block_scan(long long v, long long *warp_sum, long long &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += u;
  }
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    long long w = warp_sum[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, w, d);
      if (lane >= d) w += u;
    }
    warp_sum[lane] = w;
  }
  __syncthreads();
  const long long before = warp > 0 ? warp_sum[warp - 1] : 0;
  total = warp_sum[kPlanWarps - 1];
  __syncthreads();
  return before + inc - v;
}

__global__ void __launch_bounds__(kPlanThreads) seqs_plan_kernel(const PlanArgs a) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ int32_t pre[];  // [n + 1] entries before request i, pieces without keys among them
  __shared__ long long warp_sum[kPlanWarps];
  const int tid = threadIdx.x, n = (int)a.n, tq = a.g.tq, bk = a.g.bk;
  // 1. lengths, clamped to the tensors (a length that does not fit is reported), and the tiles of work
  long long w = 0;
  bool back = false;
  for (int b = tid; b < n; b += kPlanThreads) {
    const Request r = request_of(a.lens, b, a.err);
    const int q = r.q, kv = r.kv, nt = (q + tq - 1) / tq;
    back |= r.back;
    a.req[2 * b] = make_int4(r.q0, q, kv, r.k0);
    int longest = 0;
    if (nt > 0) {
      const TileRange f = unit_tiles(kv - q, min(tq, q), kv, bk, a.causal, a.window);
      const TileRange l = unit_tiles(kv - q + (nt - 1) * tq, q - (nt - 1) * tq, kv, bk, a.causal, a.window);
      // without a window a unit's tiles never shrink with its position; a window bounds them
      longest = max(f.e - f.a, l.e - l.a);
      if (a.window > 0) {
        const long long most = ((long long)a.window + tq + 2 * bk - 3) / bk + 1;
        longest = (int)min(most, (long long)(kv + bk - 1) / bk);
      }
      w += (long long)nt * (f.e - f.a + l.e - l.a + 1) / 2;
    }
    a.req[2 * b + 1] = make_int4(nt, longest, 1, 0);
  }
  long long work;
  block_scan(w, warp_sum, work);
  work *= a.Hk;
  if (__syncthreads_or(back)) {
    if (tid == 0) {
      a.counters[0] = a.counters[1] = a.counters[2] = a.counters[3] = 0;
    }
    return;
  }
  // 2. tiles a piece: two thirds of an even share, doubled until the partial results fit their space
  long long cut = max((long long)a.g.min_tiles, (2 * work + 3 * a.g.ctas - 1) / (3 * a.g.ctas));
  long long slots, entries;
  for (;; cut *= 2) {
    long long s_carry = 0, e_carry = 0;
    for (int c0 = 0; c0 < n; c0 += kPlanThreads) {
      const int b = c0 + tid;
      long long es = 0, ss = 0;
      int4 r = {0, 0, 0, 0};
      if (b < n) {
        r = a.req[2 * b + 1];
        // (y is the longest unit's tiles on the first pass, w its copy for the next)
        const int longest = r.w ? r.w : max(r.y, 1);
        const int pieces = (int)((longest + cut - 1) / cut);
        r.w = longest;
        r.z = pieces;
        r.y = (longest + pieces - 1) / pieces;
        es = (long long)a.Hk * r.x * pieces;
        ss = pieces > 1 ? es : 0;
      }
      long long et, st;
      const long long e0 = block_scan(es, warp_sum, et), s0 = block_scan(ss, warp_sum, st);
      if (b < n) {
        pre[b] = (int)(e_carry + e0);
        a.req[2 * b + 1] = r;
        // slot bases are kept beside the prefix until the cut is settled
        pre[n + 1 + b] = (int)min(s_carry + s0, (long long)INT_MAX);
      }
      s_carry += st;
      e_carry += et;
    }
    slots = s_carry;
    entries = e_carry;
    if (slots <= a.g.n_slots) break;
  }
  if (tid == 0) pre[n] = (int)entries;
  __syncthreads();
  // 3. the entries, pieces without keys left out (a unit without any key keeps one).  Where no unit
  // is cut every entry stays, in order.  Otherwise the pieces go by length, a quarter of the longest
  // at a time, each quarter in order: long pieces taken last would leave the other CTAs idle.
  const bool all = slots == 0;
  const int n_entries = (int)entries;
  auto entry = [&](int e, SeqsItem &it, SeqsMerge &mg) -> int {  // quarter of a piece, -1: no keys of it
    int lo = 0, hi = n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= e) lo = mid; else hi = mid;
    }
    const int4 r0 = a.req[2 * lo], r1 = a.req[2 * lo + 1];
    const int nt = r1.x, pieces = r1.z, per = r1.y;
    int x = e - pre[lo];
    const int t = nt - 1 - x % nt;
    x /= nt;
    const int s = x % pieces, h = x / pieces;
    it.b = lo;
    it.h = h;
    it.nt = min(tq, r0.y - t * tq);
    it.qrow0 = r0.x + t * tq;
    it.pos0 = r0.z - r0.y + t * tq;
    it.kv = r0.z;
    it.krow0 = r0.w;
    const TileRange u = unit_tiles(it.pos0, it.nt, it.kv, bk, a.causal, a.window);
    const int tiles = u.e - u.a;
    const int mine = max(1, (tiles + per - 1) / per);  // pieces of this unit
    it.key0 = (u.a + s * per) * bk;
    it.key1 = tiles > 0 ? min((u.a + min((s + 1) * per, tiles)) * bk, u.hi) : it.key0;
    const int slot0 = pre[n + 1 + lo] + h * pieces * nt + t;
    it.slot = mine > 1 ? slot0 + s * nt : -1;
    it.pad[0] = it.pad[1] = 0;
    mg.h = h;
    mg.nt = s == 0 && mine > 1 ? it.nt : 0;  // tokens of a unit to merge, told by its first piece
    mg.qrow0 = it.qrow0;
    mg.slot0 = slot0;
    mg.slot1 = slot0 + nt;
    mg.stride = nt;
    mg.nseg = mine;
    if (s >= mine) return -1;
    const long long len = min(per, tiles - s * per);
    return 3 - (int)min(3ll, 4 * len / (cut + 1));
  };
  SeqsItem it;
  SeqsMerge mg;
  if (all) {
    for (int e = tid; e < n_entries; e += kPlanThreads) {
      entry(e, it, mg);
      a.items[e] = it;
    }
    if (tid == 0) {
      a.counters[0] = a.counters[2] = a.counters[3] = 0;
      a.counters[1] = (unsigned)n_entries;
    }
    return;
  }
  // counts of the four quarters, 16 bits each in a scan over 1,024 entries
  int at[4] = {0, 0, 0, 0}, n_merges = 0, n_groups = 0;
  for (int c0 = 0; c0 < n_entries; c0 += kPlanThreads) {
    const int e = c0 + tid, c = e < n_entries ? entry(e, it, mg) : -1;
    long long sum;
    block_scan(c < 0 ? 0ll : 1ll << (16 * c), warp_sum, sum);
#pragma unroll
    for (int i = 0; i < 3; ++i) at[i + 1] += (int)((sum >> (16 * i)) & 0xffff);
    at[0] += (int)((sum >> 48) & 0xffff);
  }
  // at[0] has counted the last quarter: the starts follow
  const int n_items = at[0] + at[1] + at[2] + at[3];
  at[2] += at[1];
  at[3] += at[2];
  at[0] = 0;
  for (int c0 = 0; c0 < n_entries; c0 += kPlanThreads) {
    const int e = c0 + tid, c = e < n_entries ? entry(e, it, mg) : -1;
    long long sum;
    const long long before = block_scan(c < 0 ? 0ll : 1ll << (16 * c), warp_sum, sum);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (c == i) a.items[at[i] + (int)((before >> (16 * i)) & 0xffff)] = it;
      at[i] += (int)((sum >> (16 * i)) & 0xffff);
    }
    // units cut, and their groups of kMergeRows rows
    const int groups = c >= 0 && mg.nt > 0 ? (mg.nt * a.g.group + kMergeRows - 1) / kMergeRows : 0;
    const long long mb = block_scan(groups > 0 ? (1ll << 32) | groups : 0ll, warp_sum, sum);
    mg.group0 = n_groups + (int)(mb & 0xffffffffll);
    if (groups > 0) a.merges[n_merges + (int)(mb >> 32)] = mg;
    n_merges += (int)(sum >> 32);
    n_groups += (int)(sum & 0xffffffffll);
  }
  if (tid == 0) {
    a.counters[0] = 0;
    a.counters[1] = (unsigned)n_items;
    a.counters[2] = (unsigned)n_merges;
    a.counters[3] = (unsigned)n_groups;
  }
}

// ---------------------------------------------------------------- merge of cut units
struct MergeArgs {
  const unsigned int *counters;
  const SeqsMerge *merges;
  const float *part_o;
  const float2 *part_ml;
  int slot_rows, group, per_cta;
  int64_t T;
  float *lse;
  View o;
};

template <typename E>
__device__ __forceinline__ E to_out(float x);
template <>
__device__ __forceinline__ float to_out<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 to_out<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half to_out<__half>(float x) { return __float2half_rn(x); }

// One warp a row, kMergeRows rows a CTA and step: with piece s holding (o_s, m_s, l_s), M = max m_s and c_s = 2^(m_s - M),
//   o = sum c_s o_s / sum c_s l_s,  lse = ln2 (M + log2 sum c_s l_s),
// pieces taken in key order.  Bound by reading the partial results, which are still in L2.
template <typename E, int D>
__device__ __forceinline__ void merge_row(const MergeArgs &a, const SeqsMerge &m, int row, int lane) {
  constexpr int EPL = D / 32;
  auto slot = [&](int s) -> int64_t { return s == 0 ? m.slot0 : m.slot1 + (s - 1) * m.stride; };
  // lane s holds piece s's max and sum; 32 pieces at a time
  float M = -INFINITY, l = 0.f, o[EPL];
#pragma unroll
  for (int e = 0; e < EPL; ++e) o[e] = 0.f;
#pragma unroll 1
  for (int s0 = 0; s0 < m.nseg; s0 += 32) {
    const int n = min(32, m.nseg - s0);
    const float2 ml = lane < n ? a.part_ml[slot(s0 + lane) * a.slot_rows + row] : make_float2(-INFINITY, 0.f);
    float mx = ml.x;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    mx = fmaxf(M, mx);
    const float keep = M == -INFINITY ? 0.f : exp2f(M - mx);  // of the pieces before these
    M = mx;
    l *= keep;
#pragma unroll
    for (int e = 0; e < EPL; ++e) o[e] *= keep;
    const float c_mine = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
#pragma unroll 4
    for (int s = 0; s < n; ++s) {
      const float c = __shfl_sync(0xffffffffu, c_mine, s);
      l = fmaf(__shfl_sync(0xffffffffu, ml.y, s), c, l);
      const float *src = a.part_o + (slot(s0 + s) * a.slot_rows + row) * D + lane * EPL;
      if constexpr (EPL == 4) {
        const float4 v = *reinterpret_cast<const float4 *>(src);
        o[0] = fmaf(v.x, c, o[0]);
        o[1] = fmaf(v.y, c, o[1]);
        o[2] = fmaf(v.z, c, o[2]);
        o[3] = fmaf(v.w, c, o[3]);
      } else {
        const float2 v = *reinterpret_cast<const float2 *>(src);
        o[0] = fmaf(v.x, c, o[0]);
        o[1] = fmaf(v.y, c, o[1]);
      }
    }
  }
  const float inv = l == 0.f ? 0.f : 1.0f / l;  // a row that sees no key: zeros, lse = -inf
  const int head = m.h * a.group + row % a.group;
  const int64_t tok = m.qrow0 + row / a.group;
  E *dst = reinterpret_cast<E *>(const_cast<void *>(a.o.ptr)) + head * a.o.sH + tok * a.o.sS + lane * EPL * a.o.sD;
#pragma unroll
  for (int e = 0; e < EPL; ++e) dst[e * a.o.sD] = to_out<E>(o[e] * inv);
  if (a.lse && lane == 0) a.lse[head * a.T + tok] = l == 0.f ? -INFINITY : 0.69314718055994531f * (M + log2f(l));

}

template <typename E, int D>
__global__ void __launch_bounds__(32 * kMergeRows) seqs_merge_kernel(const MergeArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  if (a.per_cta) {  // at most one cut unit begins in each CTA of the attention kernel
    const SeqsMerge m = a.merges[blockIdx.x];
    if (m.nseg < 2) return;
    for (int row = blockIdx.y * kMergeRows + (threadIdx.x >> 5); row < m.nt * a.group; row += gridDim.y * kMergeRows)
      merge_row<E, D>(a, m, row, lane);
    return;
  }
  // this CTA's even share of the groups of kMergeRows rows, found by one search of the list
  const int n_merges = (int)a.counters[2], n_groups = (int)a.counters[3];
  const int per = (n_groups + (int)gridDim.x - 1) / (int)gridDim.x;
  const int g0 = (int)blockIdx.x * per, g1 = min(g0 + per, n_groups);
  if (g0 >= g1) return;
  int i = 0;  // the last entry whose groups start at or before g0: 32 entries looked at a step
  for (int n = n_merges; n > 1;) {
    const int step = (n + 31) / 32, at = i + lane * step;
    const unsigned before = __ballot_sync(0xffffffffu, lane * step < n && a.merges[at].group0 <= g0);
    const int last = 31 - __clz(before);
    i += last * step;
    n = min(step, n - last * step);
  }
  SeqsMerge m = a.merges[i];
  for (int g = g0; g < g1; ++g) {
    while (g - m.group0 >= (m.nt * a.group + kMergeRows - 1) / kMergeRows) m = a.merges[++i];
    const int row = (g - m.group0) * kMergeRows + (threadIdx.x >> 5);
    if (row >= m.nt * a.group) continue;
    merge_row<E, D>(a, m, row, lane);
  }
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

SeqsSpace seqs_space(const SeqsGeom &g, int64_t n, int64_t T, int64_t Hk, int64_t D) {
  SeqsSpace s;
  // a piece for every unit, and the pieces of cut units beyond their first
  s.max_items = (T / g.tq + n) * Hk + g.n_slots;
  size_t at = 0;
  s.counters = at;
  at += 256;
  s.req = at;
  at = up(at + (size_t)n * 32);
  s.items = at;
  at = up(at + (size_t)s.max_items * sizeof(SeqsItem));
  s.merges = at;
  at = up(at + (size_t)g.n_slots * sizeof(SeqsMerge));
  s.part_ml = at;
  at = up(at + (size_t)g.n_slots * (size_t)g.slot_rows * 8);
  s.part_o = at;
  at = up(at + (size_t)g.n_slots * (size_t)g.slot_rows * (size_t)D * 4);
  s.total = at;
  return s;
}

cudaError_t seqs_plan_prepare() {
  return cudaFuncSetAttribute(seqs_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (2 * kMaxSeqs + 2) * 4);
}

cudaError_t launch_seqs_plan(const SeqsArgs &a, const SeqsGeom &g, const SeqsSpace &s, cudaStream_t st) {
  uint8_t *ws = static_cast<uint8_t *>(a.ws);
  PlanArgs p;
  p.lens = seqs_lens(a);
  p.n = a.n;
  p.Hk = (int)a.k.H;
  p.causal = a.causal;
  p.window = a.window;
  p.g = g;
  p.counters = reinterpret_cast<unsigned int *>(ws + s.counters);
  p.req = reinterpret_cast<int4 *>(ws + s.req);
  p.items = reinterpret_cast<SeqsItem *>(ws + s.items);
  p.merges = reinterpret_cast<SeqsMerge *>(ws + s.merges);
  p.err = a.err;
  const size_t smem = (size_t)(2 * a.n + 2) * 4;
  return launch_pdl(seqs_plan_kernel, dim3(1), dim3(kPlanThreads), smem, st, p);
}

cudaError_t launch_seqs_merge(const SeqsArgs &a, const SeqsGeom &g, const SeqsSpace &s, cudaStream_t st) {
  const uint8_t *ws = static_cast<const uint8_t *>(a.ws);
  MergeArgs m;
  m.counters = reinterpret_cast<const unsigned int *>(ws + s.counters);
  m.merges = reinterpret_cast<const SeqsMerge *>(ws + s.merges);
  m.part_o = reinterpret_cast<const float *>(ws + s.part_o);
  m.part_ml = reinterpret_cast<const float2 *>(ws + s.part_ml);
  m.slot_rows = g.slot_rows;
  m.group = g.group;
  m.per_cta = g.stream;
  m.T = a.q.S;
  m.lse = a.lse;
  m.o = a.o;
  // without a list of cut units, one CTA for each that may be, more where requests have many rows: of one a
  // token up to 8, and of one for each kMergeRows rows up to 32, the larger (one tree of 64 nodes over 30k keys,
  // 256 rows a unit: 66 us with 8, 55 with 32; decoding, where one a token was all, with 64 query heads to a key
  // head: one request over 30k keys 104 -> 36, 64 over 4k 60 -> 50, 8 of two tokens over 8k 61 -> 33; 32 to one: 64
  // over 8k 121 -> 115, 4 over 65k 86 -> 74; up to 8 to one the same)
  const int64_t tokens = (a.q.S + a.n - 1) / a.n, each = (tokens * g.group + kMergeRows - 1) / kMergeRows;
  const int64_t few = tokens < 8 ? tokens : 8, many = each < 32 ? each : 32;
  const dim3 grid = g.stream ? dim3((unsigned)g.ctas, (unsigned)(few > many ? few : many)) : dim3((unsigned)(8 * g.ctas));
  const dim3 threads(32 * kMergeRows);
  if (a.o.D == 128) {
    if (a.o.dtype == FM_F32) return launch_pdl(seqs_merge_kernel<float, 128>, grid, threads, 0, st, m);
    if (a.o.dtype == FM_BF16) return launch_pdl(seqs_merge_kernel<__nv_bfloat16, 128>, grid, threads, 0, st, m);
    return launch_pdl(seqs_merge_kernel<__half, 128>, grid, threads, 0, st, m);
  }
  if (a.o.dtype == FM_F32) return launch_pdl(seqs_merge_kernel<float, 64>, grid, threads, 0, st, m);
  if (a.o.dtype == FM_BF16) return launch_pdl(seqs_merge_kernel<__nv_bfloat16, 64>, grid, threads, 0, st, m);
  return launch_pdl(seqs_merge_kernel<__half, 64>, grid, threads, 0, st, m);
}

}  // namespace fm
