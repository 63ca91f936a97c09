// fm_seqs_tc.cuh -- attention over requests of different lengths on the tensor cores (sm_103a):
// packed prompts, chunks over a paged cache, and decoding, for bf16 and fp16, D = 64 or 128.
//
//   S = Q K^T   tcgen05.mma, Q and K from swizzled shared memory (TMA), fp32 in tensor memory
//   P           online softmax of the rows (running max, rescaled lazily), rounded to the inputs' type
//               over S in tensor memory; sums in fp32 registers, of the weights before they are rounded
//   O += P V    tcgen05.mma, P from tensor memory, V from shared memory
//
// Rows.  A tile's 128 rows are floor(128 / G) tokens x the G query heads of one key head, token by
// token, so that the heads that share a key head read it once and a decoding request fills G rows
// with one pass over its keys.  One 3-D TMA box {64, G, tokens} per 64 columns gathers a tile.
// Keys.  A tile's 128 keys are one TMA box (packed, or pages of 128 keys and more: 64-column panels
// of 128 rows) or one box a page, one lane of the producer warp a box.  A page's box brings its
// 64-column panels for each 8 keys together ({64, 8, panels, page_size / 8}), so that a tile's
// groups of 8 keys are evenly spaced whatever the page size, which a matrix descriptor needs: one
// box a page and panel was bound by the number of boxes (decode batch of 64 over 8k keys, 16-key pages:
// 176 us against 149; 32-key pages 149 both ways, the rate of HBM).  Pages past the request's end are asked for at a page that
// does not exist, which TMA fills with zeros, and so are pages before the unit's window.
// Work.  A CTA a SM takes pieces from the list in order (a counter), or, where requests have few
// queries, an even run of all units' key tiles.  A piece is a unit of queries
// -- two row tiles, or one when its tokens fit one (decoding, the rest of a chunk) -- against a
// range of keys.  The tensor core always alternates between two softmax groups of four warps:
//   two row tiles   group g has row tile g, both against the same key tile
//   one row tile    group g has the key tiles of parity g, with an O and a max of its own, joined
//                   at the end: a decoding request's tiles go through both groups at once
// MMA order for step s of a piece (group s mod 2):  S(s), P V(s - 1): one group's softmax runs
// under the other's two MMAs.
// 12 warps: 0 K/V producer, 1 MMA issuer (and TMEM), 2 zeroes V rows past the request's end or before
// the window (they meet p = 0, but may hold NaN), 3 fetches work and loads its Q, 4-7 and 8-11 softmax.
// TMEM: S0 [0,128) S1 [128,256) O0 [256,256+D) O1 [384,384+D).
// Measured (us a call, plan and merge with it): decode batch of 64 over 8k keys (40 / 8 heads) 130, 84 %
// of the copy rate; 24 prompts of up to 4,096 676, one of 33,001 7,957 (1,400 TFLOP/s, 73 % of the
// measured burst rate).  Decoding is bound by HBM; prompts by the cycle of a group's softmax and its MMAs
// (1.66 us a tile pair, of which 1.33 are MMAs), and by about 5 us of a unit's start and end.
// (Figures of one kernel against another below are of calls made alone, L2 flushed before each.)
// Every wait is bounded; on expiry the kernel records it and returns, as the chunk kernel does.
//
// P has 16 bits because the operands of a tcgen05.mma of 16-bit kind share one type, and V has the
// inputs'; as tf32, V would have to be converted and the MMA would run at half the rate.  Each weight is off
// by at most half a step (2^-8 relative in bf16, 2^-11 in fp16), o by no more than that of sum p |v|: over whole
// outputs 0.0020 to 0.0023 (2-norm, bf16) and 0.0003 (fp16) from 64 bits, where rounding o alone leaves
// 0.0016 to 0.0017 and 0.0002.
//
// TREE (fm_attn_tree): of a request's new tokens a row sees those that its mask row names.  Only how a
// tile is masked differs (mask_tree), in the one or two tiles at a unit's end that hold new tokens.
#pragma once

#include <cudaTypedefs.h>
#include <limits.h>
#include <string.h>

#include <mutex>

#include "fm_seqs.cuh"
#include "fm_tc.cuh"

namespace fm {
namespace {

constexpr int kThreads = 384;
constexpr int kPanel = 128 * 128;  // 128 rows of 64 16-bit columns: one 128-byte swizzle span

template <typename E, int D, bool GROUPED>
struct Cfg {
  static constexpr int PN = D / 64;          // panels of a tile
  // bytes between a K or V tile's panels, and between its groups of 8 keys (GROUPED: see encode_pages)
  static constexpr int kPanelStep = GROUPED ? 1024 : kPanel, kGroupStep = GROUPED ? 1024 * PN : 1024;
  static constexpr int kTile = PN * kPanel;  // bytes
  static constexpr int NS = 10 / PN;         // K/V ring: 160 KiB
  static constexpr int offQ = 0;
  static constexpr int offKV = 2 * kTile;
  static constexpr int offStat = offKV + NS * kTile;  // (max, sum) of group 1's rows
  static constexpr int offItems = offStat + 128 * 8;
  static constexpr int offBar = offItems + 2 * (int)sizeof(SeqsItem);
  // barriers
  static constexpr int QFull = 0, QEmpty = 2, SFull = 4, PReady = 6, ODone = 8, ItemFull = 10, ItemEmpty = 12, VNeed = 14,
                       VFix = 15, Stat = 16, EpiDone = 17, Want = 18, Drain = 19, KVFull = 20, KVEmpty = KVFull + NS,
                       kBars = KVEmpty + NS;
  static constexpr int offTmem = offBar + kBars * 8;
  static constexpr int offAbort = offTmem + 8;
  static constexpr int kSmem = offAbort + 8 + 1024;  // slack for aligning the base
  static_assert(kSmem <= 232448, "shared memory of an SM");
  static constexpr bool bf16 = std::is_same<E, __nv_bfloat16>::value;
  static constexpr uint32_t idescQK = idesc_f16(128, 128, false, bf16);  // K [keys, D]: K-major
  static constexpr uint32_t idescPV = idesc_f16(128, D, true, bf16);     // V [keys, D]: MN-major
};
// How a call's work is dealt out: even runs cut by the kernel (requests of few queries), the work list,
// and the work list of long prompts at D = 64.
enum : int { kStream, kList, kLong };
constexpr int kItemReaders = 11;  // arrivals that free an item slot: warps 0, 1, 2 and the 8 softmax warps

struct Maps {
  CUtensorMap q, k, v;
};
struct Params {
  int group, tq1;  // heads of a key head, tokens of a row tile
  uint32_t inv_group;  // ceil(2^16 / group): row * inv_group >> 16 is row / group for the rows of a tile
  int wide;            // o's rows are 32-byte aligned
  int causal, window;
  float alpha;
  int paged, ps, box_rows, num_pages;
  int page_groups;  // groups of 8 keys from one page to the next (GROUPED)
  const int32_t *table;
  int64_t table_stride;
  unsigned int *counters;
  const SeqsItem *items;
  SeqsMerge *merges;
  SeqsLens lens;
  int n, Hk;
  float *part_o;
  float2 *part_ml;
  int slot_rows;
  void *out;
  int out_f32;
  int64_t osH, osS;
  float *lse;
  int64_t T;
  const uint32_t *mask;  // TREE: rows of mask_words words, mask_stride apart
  int mask_words;
  int64_t mask_stride;
  unsigned int *err;
  unsigned long long timeout_ns;
};

__device__ __forceinline__ void prefetch_map(const CUtensorMap *tm) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tm)) : "memory");
}
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *tm, uint32_t bar, int c0, int c1, int c2, int c3,
                                            int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *tm, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// The code that runs once a piece (masks, epilogue) is kept in short loops: straight-line code that
// is not in the instruction cache takes longer to fetch than to run (64 causal prompts of 512:
// 227 -> 183 us when it was changed, 140 now).

// Online softmax of one S tile for this thread's row, as softmax_online_tile, but exponentiating in
// a loop over the two halves of the columns (LOOPS = 1) for the same reason: 203 -> 185 us for 32
// prompts of 1,024 (16 / 4 heads, D = 128), 727 -> 674 us for 24 of up to 4,096 (40 / 8 heads), and no
// loss at 33k (7.82 and 7.78 ms).  At D = 64 a tile has half the MMA time to hide it, and long
// prompts do better unrolled (LOOPS = 2), which packed prompts of 4,096 and more on average take: one of
// 20,000 2.89 -> 2.51 ms, of 6,000 323 -> 289 us, of 4,096 180 -> 165; 4 of 4,096 each 575 -> 524, 16 of
// them 2,143 -> 1,948.  Below, gains end between 2,048 (4 of them 191 -> 183 us, 16 628 -> 612) and 1,024 (4 of
// them 83 -> 84); of unequal lengths, 16 of up to 2,048 lose (162 -> 166), 4 of up to 4,096 gain (232 -> 219).
// The bound on the mean lies where every mix that was measured gains.
template <typename E, int D, int LOOPS>
__device__ __forceinline__ void softmax_tile(uint32_t tS, uint32_t tO, float alpha, bool have_o, float &run, float (&l)[4]) {
  uint32_t sa[32], sb[32], pk[16];
  float mx = -INFINITY;
#pragma unroll
  for (int h = 0; h < 128; h += 64) {
    tmem_ld32_async(tS + h, sa);
    tmem_ld32_async(tS + h + 32, sb);
    tmem_ld_wait(sa);
    tmem_reg_tie(sb);
    mx = max64(sa, sb, mx);
  }
  const float zmax = mx * alpha;
  const bool need = run == -INFINITY || zmax > run + kLazyRescale;
  const bool any = __any_sync(0xffffffffu, need);
  float sc = 1.0f;
  if (any) {
    const float nr = need ? fmaxf(run, zmax) : run;
    // O holds earlier tiles only with have_o, and nothing but zeros while run is -inf
    if (have_o && need) sc = run == -INFINITY ? 0.f : ex2(run - nr);
    run = nr;
#pragma unroll
    for (int i = 0; i < 4; ++i) l[i] *= sc;
  }
  const float nbias = run == -INFINITY ? 0.f : -(run - p_bias<E>());
  const uint64_t a2 = f2_pack(__float_as_uint(alpha), __float_as_uint(alpha));
  const uint64_t nb2 = f2_pack(__float_as_uint(nbias), __float_as_uint(nbias));
  uint64_t acc0 = 0, acc1 = 0;
  tmem_ld32_async(tS, sa);
#pragma unroll LOOPS
  for (int h = 0; h < 2; ++h) {
    tmem_ld_wait(sa);
    tmem_ld32_async(tS + 64 * h + 32, sb);
    exp_chunk_full<E, 0>(sa, a2, nb2, acc0, acc1, pk);
    tmem_st16(tS + 32 * h, pk);  // P columns lie in S columns already read
    tmem_ld_wait(sb);
    if (h == 0) tmem_ld32_async(tS + 64, sa);
    exp_chunk_full<E, 0>(sb, a2, nb2, acc0, acc1, pk);
    tmem_st16(tS + 32 * h + 16, pk);
  }
  float x0, x1, y0, y1;
  f2_unpack(acc0, x0, x1);
  f2_unpack(acc1, y0, y1);
  l[0] += x0;
  l[1] += x1;
  l[2] += y0;
  l[3] += y1;
  if (any && have_o) {
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
      tmem_ld32(tO + c, sa);
#pragma unroll
      for (int e = 0; e < 32; ++e) sa[e] = __float_as_uint(__uint_as_float(sa[e]) * sc);
      tmem_st32(tO + c, sa);
    }
  }
}

// Bits [0, n) set, for n of any sign.
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u); }

// Scores outside [lo, hi) of the row's keys become -inf; kb is the tile's first key, and the
// warp's rows all see [max_lo, min_hi), so that column blocks inside it are left alone.
__device__ __noinline__ void mask_rows(uint32_t tS, int kb, int lo, int hi, int max_lo, int min_hi) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c, tS += 32, kb += 32) {
    if (kb >= max_lo && kb + 32 <= min_hi) continue;
    const uint32_t keep = low_bits(hi - kb) & ~low_bits(lo - kb);
    uint32_t s[32];
    tmem_ld32(tS, s);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (!((keep >> e) & 1u)) s[e] = 0xff800000u;  // -inf
    tmem_st32(tS, s);
  }
  tmem_st_wait();
}

// The same where new tokens are seen by the row's mask: `bits` has `words` words (0: no row), its bit 0
// is key `base`.  The warp's rows all see every key before min_hi.
__device__ __noinline__ void mask_tree(uint32_t tS, int kb, int hi, int min_hi, int base, const uint32_t *bits, int words) {
#pragma unroll 1
  for (int c = 0; c < 4; ++c, tS += 32, kb += 32) {
    if (kb + 32 <= min_hi) continue;
    const uint32_t keep = low_bits(hi - kb) & tree_bits(bits, words, kb - base);
    uint32_t s[32];
    tmem_ld32(tS, s);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if (!((keep >> e) & 1u)) s[e] = 0xff800000u;  // -inf
    tmem_st32(tS, s);
  }
  tmem_st_wait();
}

// 32 bytes of a row in one store (wide: 32-byte aligned) or two.
__device__ __forceinline__ void store32(uint8_t *dst, const uint32_t (&w)[8], bool wide) {
  if (wide)
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  else {
    *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    *reinterpret_cast<uint4 *>(dst + 16) = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
// 32 columns of this lane's row to memory, as 16-bit elements or fp32.  Whole 32-byte sectors, lane by
// lane: few instructions, and the stores drain while the next piece starts.
template <typename E>
__device__ __forceinline__ void store_row(uint8_t *dst, const float (&x)[32], bool f32, bool wide) {
  uint32_t w[8];
  if (f32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(x[8 * i + e]);
      store32(dst + 32 * i, w, wide);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = pack_half<E>(x[16 * i + 2 * e], x[16 * i + 2 * e + 1]);
      store32(dst + 32 * i, w, wide);
    }
  }
}

// A descriptor's upper half: stride of 8 rows in 16-byte units, version, 128-byte swizzle.
__device__ __forceinline__ uint64_t desc(uint32_t step, uint32_t lo) {
  return ((uint64_t)(step | (1u << 14) | (2u << 29)) << 32) | lo;
}

// S = Q K^T of one tile pair, then the arrival at `done`; a, b: lower halves of Q's and K's descriptors.
// Unrolled with constant steps: an MMA has to be issued in less time than it runs, and with steps
// in registers or a loop around it it is not (1.66 -> 2.4 us a tile).
template <typename C>
__device__ __forceinline__ void mma_scores(uint32_t tS, uint32_t a, uint32_t b, uint32_t done) {
#pragma unroll
  for (int kk = 0; kk < 4 * C::PN; ++kk) {
    const uint32_t o = (uint32_t)((kk & 3) * 2);
    mma_ss(tS, desc(64, a + o + (uint32_t)((kk >> 2) * (kPanel >> 4))),
           desc(C::kGroupStep >> 4, b + o + (uint32_t)((kk >> 2) * (C::kPanelStep >> 4))), C::idescQK, kk > 0);
  }
  mma_commit(done);
}
// O (+)= P V of one tile; b: lower half of V's descriptor.
template <typename C>
__device__ __forceinline__ void mma_output(uint32_t tO, uint32_t tP, uint32_t b, uint32_t acc) {
  mma_ts(tO, tP, desc(C::kGroupStep >> 4, b), C::idescPV, acc);
#pragma unroll
  for (int kk = 1; kk < 8; ++kk)
    mma_ts(tO, tP + kk * 8, desc(C::kGroupStep >> 4, b + (uint32_t)(kk * 2 * (C::kGroupStep >> 4))), C::idescPV, 1);
}

// ---------------------------------------------------------------- one even run per CTA
// Calls of few queries a request (decoding) take no work list: the units in order of request, key
// head and queries, each as long as its key tiles take, are one line, and CTA c takes the
// c-th of equal parts.  A unit that a boundary cuts leaves partial results: a CTA has at most one
// piece that continues a unit (slot 2c) and one that begins a unit and does not end it (2c + 1).
// The line's measure, in about 0.35 us: a key tile of a unit of one row tile (streamed from HBM) and
// of two (bound by the tensor core and the exponentials), and a unit's start and end.
constexpr int kTileCost1 = 4, kTileCost2 = 5, kUnitCost1 = 12, kUnitCost2 = 20;
constexpr int kLeastRun = 12;  // shorter runs would cost more to merge than they save (none is shorter than a tile)
// (trees, whose units have many rows to store and merge for few tiles: captured, one of 26 over 900 keys 17.4 us
// with 12, 16.4 with 8, 16.7 with 6, 20.4 with 24; one of 8 over 300 13.7, 11.8, 11.7, 13.3; one of 60 24.3, 22.8,
// 23.1, 27.0.  A line is at least one unit, 12, so that its parts are at least 8 * 12 / 19 = 5 long, as a tile of
// two row tiles is: every part of a unit's tiles holds the start of one.  Parts of 6 would not.)
constexpr int kLeastRunTree = 8;
static_assert(kLeastRunTree * kUnitCost1 / (kUnitCost1 + kLeastRunTree - 1) >= kTileCost2, "no run is shorter than a tile");

// This CTA's part [x0, x1) of the line, and the unit that x0 falls in: (b, h, t), starting at u0.
struct StreamRun {
  int total, x0, x1, u0;
  int parts, b, h, t;
  Request req;
};
// The line is measured in 32 bits, sums stopping at kMostLine: a call of so much (4.3e8 key tiles of units of
// two row tiles, 5.4e8 of one: some 5 s of the whole GPU by the measure above) is refused as lengths that do
// not fit.
constexpr int kMostLine = 0x7fff0000;

__device__ __forceinline__ int unit_cost(const Params &p, const Request &r, int t) {
  const int tq = 2 * p.tq1;
  const int nt = min(tq, r.q - t * tq);
  const TileRange u = unit_tiles(r.kv - r.q + t * tq, nt, r.kv, 128, p.causal, p.window);
  return nt > p.tq1 ? (u.e - u.a) * kTileCost2 + kUnitCost2 : (u.e - u.a) * kTileCost1 + kUnitCost1;
}
__device__ __forceinline__ long long request_cost(const Params &p, const Request &r) {  // of one key head
  long long c = 0;
#pragma unroll 1
  for (int t = 0; t * 2 * p.tq1 < r.q; ++t) c += unit_cost(p, r, t);
  return c;
}
// a * b / c for a line of length a: 32-bit division where the product fits (b < 256)
__device__ __forceinline__ int part_of(int a, int b, int c) {
  if (a < (1 << 24)) return (int)(((unsigned)a * (unsigned)b) / (unsigned)c);
  return (int)((long long)a * b / c);
}

// Every thread of the CTA: sums the requests' costs, a run of requests a thread, in one scan, and
// the thread whose requests hold x0 finds the unit.  A few dependent steps after one round of
// loads, in as little code as can be: it stands before the first tile of every call.
__device__ __forceinline__ void stream_run(const Params &p, int least, int *warp_sum, StreamRun *out) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = (p.n + kThreads - 1) / kThreads, b0 = tid * each, b1 = min(b0 + each, p.n);
  unsigned int *err = blockIdx.x == 0 ? p.err : nullptr;
  long long sum = 0, per_head = 0;
  bool refuse = false;
  Request r = {0, 0, 0, 0, false};
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    r = request_of(p.lens, b, err);
    per_head = request_cost(p, r);
    sum += per_head * p.Hk;
    refuse |= r.back;
  }
  auto plus = [](int x, int y) { return (int)min((unsigned)x + (unsigned)y, (unsigned)kMostLine); };
  const int mine = (int)min(sum, (long long)kMostLine);
  int inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc = plus(inc, u);
  }
  if (lane == 31) warp_sum[warp] = inc;
  // no unit begins in this CTA's run until the walk says so: a wait that gives up before that leaves
  // no stale entry for the merge
  if (tid == 0) p.merges[blockIdx.x].nseg = 0;
  const bool none = __syncthreads_or(refuse);
  int start = inc - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int x = warp_sum[w];
    if (w < warp) start = plus(start, x);
    total = plus(total, x);
  }
  if (total == kMostLine && err && tid == 0 && atomicCAS(err, 0u, (unsigned)kDevErrLength) == 0u)
    err[1] = err[2] = err[3] = err[4] = 0u;
  if (none || total == kMostLine) total = 0;
  const int parts = max(1, min((int)gridDim.x, (total + least - 1) / least)), c = blockIdx.x;
  int x0 = 0, x1 = 0;
  if (c < parts) {
    x0 = part_of(total, c, parts);
    x1 = part_of(total, c + 1, parts);
  }
  if (tid == 0) {
    out->total = total;
    out->parts = parts;
    out->x0 = x0;
    out->x1 = x1;
  }
  if (x0 < x1 && start <= x0 && x0 < start + mine) {
    int b = b0;
    if (each > 1)
#pragma unroll 1
      for (;; ++b) {
        r = request_of(p.lens, b, nullptr);
        per_head = request_cost(p, r);
        if (x0 < start + (int)per_head * p.Hk) break;
        start += (int)per_head * p.Hk;
      }
    const int h = (unsigned)(x0 - start) / (unsigned)per_head;
    start += h * (int)per_head;
    int t = 0;
#pragma unroll 1
    for (int u; start + (u = unit_cost(p, r, t)) <= x0; ++t) start += u;
    out->b = b;
    out->h = h;
    out->t = t;
    out->u0 = start;
    out->req = r;
  }
  __syncthreads();
}

// One thread: the run's pieces in order.
struct StreamWalk {
  StreamRun r;

  // The next piece; false when the run is at its end.  Writes the CTA's merge entry, if a unit begins
  // in its run and does not end there.
  __device__ __forceinline__ bool next(const Params &p, SeqsItem &it) {
    const int tq = 2 * p.tq1;
    bool found = false;
    while (!found && r.x0 < r.x1 && r.u0 < r.x1) {
      const int nt = min(tq, r.req.q - r.t * tq), pos0 = r.req.kv - r.req.q + r.t * tq;
      const TileRange u = unit_tiles(pos0, nt, r.req.kv, 128, p.causal, p.window);
      const int tiles = u.e - u.a;
      // a tile belongs to the run that holds its start (runs are longer than a tile)
      const int cost = nt > p.tq1 ? kTileCost2 : kTileCost1;
      const int from = r.x0 > r.u0 ? (r.x0 - r.u0 + cost - 1) / cost : 0, to = min(tiles, (r.x1 - r.u0 + cost - 1) / cost);
      found = from < to || (tiles == 0 && from == 0);
      if (found) {
        it.b = r.b;
        it.h = r.h;
        it.nt = nt;
        it.qrow0 = r.req.q0 + r.t * tq;
        it.pos0 = pos0;
        it.kv = r.req.kv;
        it.krow0 = r.req.k0;
        it.key0 = (u.a + from) * 128;
        it.key1 = tiles > 0 ? min((u.a + to) * 128, u.hi) : it.key0;
        const bool whole = from == 0 && to >= tiles;
        it.slot = whole ? -1 : 2 * (int)blockIdx.x + (from == 0 ? 1 : 0);
        if (!whole && from == 0) {
          // the CTA that holds the unit's last tile: the last c with total * c / parts <= its place
          const int end = r.u0 + (tiles - 1) * cost + 1;  // one past that tile's start
          const int last = r.total < (1 << 24) ? (int)(((unsigned)end * (unsigned)r.parts - 1u) / (unsigned)r.total)
                                               : (int)(((long long)end * r.parts - 1) / r.total);
          SeqsMerge m;
          m.h = r.h;
          m.nt = nt;
          m.qrow0 = it.qrow0;
          m.nseg = last - (int)blockIdx.x + 1;
          m.slot0 = it.slot;
          m.slot1 = 2 * (int)blockIdx.x + 2;
          m.stride = 2;
          m.group0 = 0;
          p.merges[blockIdx.x] = m;
        }
      }
      r.u0 += tiles * cost + (nt > p.tq1 ? kUnitCost2 : kUnitCost1);
      if (++r.t * tq >= r.req.q) {
        r.t = 0;
        if (++r.h == p.Hk) {
          r.h = 0;
          do {
            if (++r.b >= p.n) {
              r.u0 = r.x1;  // the line ends with the last request
              break;
            }
            r.req = request_of(p.lens, r.b, nullptr);
          } while (r.req.q == 0);
        }
      }
    }
    return found;
  }
};

// The rest of a wait that did not succeed at once.  Out of line and of few arguments (parity, role,
// barrier and tag in one word): the kernel has dozens of waits.
template <typename C>
__device__ __noinline__ bool wait_more(const Params &p, uint32_t base, uint32_t what) {
  volatile int *abort_flag = reinterpret_cast<volatile int *>(__cvta_shared_to_generic(base + C::offAbort));
  const uint32_t i = (what >> 16) & 0xffu;
  return wait_phase_slow(base + (uint32_t)C::offBar + 8 * i, what >> 31, abort_flag, p.timeout_ns, p.err,
                         (what >> 24) & 0x7fu, wtag((int)i, (int)(what & 0xffffu)));
}

template <typename E, int D, bool GROUPED, int MODE, bool TREE>
__global__ void __launch_bounds__(kThreads, 1)
    seqs_tc_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  using C = Cfg<E, D, GROUPED>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *gbase = smem_raw + (base - raw);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(gbase + C::offAbort);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(gbase + C::offTmem);
  SeqsItem *item_ring = reinterpret_cast<SeqsItem *>(gbase + C::offItems);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto bar = [&](int i) -> uint32_t { return base + (uint32_t)(C::offBar + 8 * i); };
  auto wait = [&](int i, uint32_t parity, unsigned code, int tag) -> bool {
    if (mbar_test(bar(i), parity)) return true;
    return wait_more<C>(p, base, parity << 31 | code << 24 | (unsigned)i << 16 | ((unsigned)tag & 0xffffu));
  };

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < C::kBars; ++i) {
      const int count = (i == C::PReady || i == C::PReady + 1 || i == C::Stat || i == C::EpiDone) ? 128
                        : (i == C::ItemEmpty || i == C::ItemEmpty + 1)                            ? kItemReaders
                                                                                                  : 1;
      mbar_init(bar(i), count);
    }
    fence_mbar_init();
    prefetch_map(&maps.q);
    prefetch_map(&maps.k);
    prefetch_map(&maps.v);
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();  // the work list, and whatever the caller's earlier kernels wrote
  pdl_trigger();
  StreamRun *run_of_cta = reinterpret_cast<StreamRun *>(gbase + C::offStat + 128);
  if constexpr (MODE == kStream) stream_run(p, TREE ? kLeastRunTree : kLeastRun, reinterpret_cast<int *>(gbase + C::offStat), run_of_cta);

  // A wait of a whole warp of which one lane polls: 32 polling lanes take the time of 32 tests.
  auto wait_warp = [&](int i, uint32_t parity, unsigned code, int tag) -> bool {
    bool ok = true;
    if (lane == 0) ok = wait(i, parity, code, tag);
    return __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
  };
  // A wait that may last as long as a piece of work, by a warp whose polling would take issue
  // slots from the softmax warps: it sleeps between looks.  (One thread.)
  auto wait_long = [&](int i, uint32_t parity, unsigned code, int tag) -> bool {
#pragma unroll 1
    for (int look = 0; look < 20000; ++look) {
      if (mbar_test(bar(i), parity)) return true;
      if (look > 16) __nanosleep(100);
    }
    return wait(i, parity, code, tag);
  };

  // The k-th piece of this CTA, read by every lane of the calling warp from the two-slot ring.
  // False when there is none left (or a wait gave up: ok says which).
  auto next_item = [&](uint32_t k, unsigned code, bool &ok, SeqsItem &it) -> bool {
    const int slot = (int)(k & 1u);
    ok = true;
    if (lane == 0) ok = wait_long(C::ItemFull + slot, (k >> 1) & 1u, code, (int)k);
    ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
    if (!ok) return false;
    __syncwarp();  // what lane 0 has waited for is visible to the others
    it = item_ring[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::ItemEmpty + slot));
    return it.b >= 0;
  };
  auto tiles_of = [](const SeqsItem &it) { return it.key1 > it.key0 ? (it.key1 - it.key0 + 127) >> 7 : 0; };
  // keys before this one are seen by no token of the piece
  auto first_seen = [&](const SeqsItem &it) { return p.window > 0 ? max(0, it.pos0 - p.window + 1) : 0; };

  if (warp == 0) {
    // ------------------------------------------------------------ K/V producer
    const int boxes = 128 / p.box_rows;  // of one tile; this lane's is its pg-th
    const int pg = lane;
    uint32_t n = 0;  // tiles loaded into the ring so far
    bool ok = true;
    SeqsItem it;
    for (uint32_t k = 0; ok && next_item(k, kDevErrTimeoutProducer, ok, it); ++k) {
      const int tiles = tiles_of(it), lo = first_seen(it);
      // coordinates of this lane's box: row and page (packed: row of the tensor, batch 0)
      auto coords = [&](int kb, int &row, int &page) {
        if (!p.paged) {
          row = it.krow0 + kb;
          page = 0;
          return;
        }
        const int key = kb + pg * p.box_rows;
        row = p.ps > 128 ? key % p.ps : 0;
        page = p.num_pages;  // past the end, before the window: zeros
        if (lane < boxes && key < it.kv && key + p.box_rows > lo) {
          const int at = key / p.ps;
          page = p.table[it.b * p.table_stride + at];
          if (page < 0 || page >= p.num_pages) {
            report_bad_page(p.err, it.b, at, page);
            page = p.num_pages;
          }
        }
      };
      int row, page;
      if (tiles > 0) coords(it.key0, row, page);
      for (int j = 0; j < tiles && ok; ++j) {
        int row_next = 0, page_next = 0;  // the next tile's table entry, asked for a tile ahead
        if (j + 1 < tiles) coords(it.key0 + (j + 1) * 128, row_next, page_next);
        for (int w = 0; w < 2 && ok; ++w, ++n) {
          const int st = (int)(n % C::NS);
          ok = wait_warp(C::KVEmpty + st, ((n / C::NS) & 1u) ^ 1u, kDevErrTimeoutProducer, j);
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(bar(C::KVFull + st), C::kTile);
          __syncwarp();
          if (lane < boxes) {
            const uint32_t dst = base + C::offKV + st * C::kTile;
            const CUtensorMap *tm = w ? &maps.v : &maps.k;
            if constexpr (GROUPED) {
              tma_load_5d(dst + pg * p.box_rows * 128 * C::PN, tm, bar(C::KVFull + st), 0, 0, 0, page * p.page_groups, it.h);
            } else if (boxes == 1) {
              tma_load_5d(dst, tm, bar(C::KVFull + st), 0, row, 0, it.h, page);
            } else {
              for (int pn = 0; pn < C::PN; ++pn)
                tma_load_5d(dst + pn * kPanel + pg * p.box_rows * 128, tm, bar(C::KVFull + st), 0, row, pn, it.h, page);
            }
          }
        }
        row = row_next;
        page = page_next;
        if (lane == 0 && j == max(tiles - 3, 0)) mbar_arrive(bar(C::Want));  // time for the next piece
      }
      if (tiles == 0 && lane == 0) mbar_arrive(bar(C::Want));
    }
    if (!ok) {
      // every copy already issued lands before the CTA can exit: the last NS loads cover the rest
      for (uint32_t i = n > C::NS ? n - C::NS : 0; i < n; ++i)
        wait_phase(bar(C::KVFull + (int)(i % C::NS)), (i / C::NS) & 1u, nullptr, p.timeout_ns, p.err, kDevErrTimeoutDrain,
                   wtag(C::KVFull, 0));
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ V rows that are to be zero
    uint32_t n = 0, fixes = 0;
    bool ok = true;
    SeqsItem it;
    for (uint32_t k = 0; ok && next_item(k, kDevErrTimeoutProducer, ok, it); ++k) {
      const int tiles = tiles_of(it);
      if (tiles == 0) continue;
      n += 2 * tiles;
      // rows of a tile's V that are to be zero: before the window in the first, past the end in the last
      auto zero_rows = [&](uint32_t v, int from, int to) {
        // the MMA warp says when that tile's V has landed, or is the next to (its stage may be rounds ahead of this warp)
        const int st = (int)(v % C::NS);
        // (every decoding request has one to wait for, and time to poll)
        if (lane == 0)
          ok = (MODE == kStream ? wait(C::VNeed, fixes & 1u, kDevErrTimeoutProducer, (int)k)
                                : wait_long(C::VNeed, fixes & 1u, kDevErrTimeoutProducer, (int)k)) &&
               wait(C::KVFull + st, (v / C::NS) & 1u, kDevErrTimeoutProducer, (int)k);
        ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
        if (!ok) return;
        ++fixes;
        __syncwarp();
        uint8_t *tile = gbase + C::offKV + st * C::kTile;
        for (int x = from * 8 + lane; x < to * 8; x += 32) {  // 16-byte words of a panel: 64 a group of 8 keys
          uint8_t *at = tile + (x >> 6) * C::kGroupStep + (x & 63) * 16;
#pragma unroll
          for (int pn = 0; pn < C::PN; ++pn) *reinterpret_cast<uint4 *>(at + pn * C::kPanelStep) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::VFix));
      };
      const int before = first_seen(it) - it.key0, valid = it.kv - (it.key0 + (tiles - 1) * 128);
      if (before > 0) zero_rows(n - 2 * tiles + 1, 0, min(before, 128));
      if (ok && valid < 128) zero_rows(n - 1, max(valid, 0), 128);
      if (!ok) break;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    // One thread, and as few instructions as can be between a group's arrival and the MMA that waits
    // for it: descriptors are sums of constants and a stage's offset (the address field of a
    // descriptor does not carry), ring positions are stepped, not divided.
    const uint32_t q_lo = ((base + C::offQ) >> 4) | (1u << 16), k_lo = ((base + C::offKV) >> 4) | (1u << 16);
    const uint32_t v_lo = ((base + C::offKV) >> 4) | ((uint32_t)(C::kPanelStep >> 4) << 16);
    int kst = 0;                      // ring stage of the next K tile, and its phase
    uint32_t kph = 0;
    uint32_t loads0 = 0, loads1 = 0;  // uses of Q slots 0 and 1
    int qs = 0;                       // Q slot of the next piece of one row tile
    uint32_t steps0 = 0, steps1 = 0;  // softmax steps of each group so far
    uint32_t fixes = 0;
    bool ok = true;
    SeqsItem it;
    auto mma_s = [&](int g, int qt, int st) {
      mma_scores<C>(tmem + g * 128, q_lo + (uint32_t)(qt * (C::kTile >> 4)), k_lo + (uint32_t)(st * (C::kTile >> 4)),
                    bar(C::SFull + g));
    };
    auto mma_pv = [&](int g, bool first, int st) {
      mma_output<C>(tmem + 256 + g * 128, tmem + g * 128, v_lo + (uint32_t)(st * (C::kTile >> 4)), !first);
    };
    auto next = [](int &st, uint32_t &ph) {
      if (++st == C::NS) {
        st = 0;
        ph ^= 1u;
      }
    };
    for (uint32_t k = 0; ok && next_item(k, kDevErrTimeoutMma, ok, it); ++k) {
      if (lane == 0 && tiles_of(it) > 0) {
        const int tiles = tiles_of(it);
        const bool dual = it.nt > p.tq1;
        // tiles with V rows that are to be zero first: the first, where keys before the window share it,
        // and the last, past the request's end (the same tile twice, if it is both)
        const bool head = first_seen(it) > it.key0, tail = it.kv - (it.key0 + (tiles - 1) * 128) < 128;
        // V of the piece's tile j has landed, and those rows are zero
        auto v_ready = [&](int j, int st, uint32_t ph) -> bool {
          if (!wait(C::KVFull + st, ph, kDevErrTimeoutMma, j)) return false;
          if constexpr (TREE) return !(tail && j == tiles - 1) || wait(C::VFix, fixes++ & 1u, kDevErrTimeoutMma, j);
          for (int f = (head && j == 0) + (tail && j == tiles - 1); f > 0; --f) {
            mbar_arrive(bar(C::VNeed));
            if (!wait(C::VFix, fixes++ & 1u, kDevErrTimeoutMma, j)) return false;
          }
          return true;
        };
        // Trees (no window, so that only a unit's last tile has such rows): warp 2 hears of the tile when its K is
        // here, and works beside the scores and the softmax (one tree of 26 over 900 keys 16.3 -> 15.3 us,
        // captured).  K's load is the one before V's, so that every earlier load of V's stage has landed, and the
        // phase of the stage that warp 2 waits for is the next to complete.
        auto k_here = [&](int j) {
          if (TREE && tail && j == tiles - 1) mbar_arrive(bar(C::VNeed));
        };
        int vst = 0;
        uint32_t vph = 0;
        if (dual) {
          ok = wait(C::QFull, loads0++ & 1u, kDevErrTimeoutMma, (int)k);
          for (int j = 0; j < tiles && ok; ++j) {
            ok = wait(C::KVFull + kst, kph, kDevErrTimeoutMma, j);
            if (!ok) break;
            k_here(j);
            tc_fence_after();
            mma_s(0, 0, kst);
            if (j == tiles - 1) mma_commit(bar(C::QEmpty));
            if (j > 0) {
              ok = wait(C::PReady + 1, steps1++ & 1u, kDevErrTimeoutMma, j);
              if (!ok) break;
              tc_fence_after();
              mma_pv(1, j == 1, vst);
              mma_commit(bar(C::KVEmpty + vst));
            } else {
              ok = wait(C::QFull + 1, loads1++ & 1u, kDevErrTimeoutMma, (int)k);
              if (!ok) break;
              tc_fence_after();
            }
            mma_s(1, 1, kst);
            mma_commit(bar(C::KVEmpty + kst));
            if (j == tiles - 1) mma_commit(bar(C::QEmpty + 1));
            next(kst, kph);
            vst = kst;
            vph = kph;
            next(kst, kph);
            ok = v_ready(j, vst, vph) && wait(C::PReady, steps0++ & 1u, kDevErrTimeoutMma, j);
            if (!ok) break;
            tc_fence_after();
            mma_pv(0, j == 0, vst);
            if (j == tiles - 1) mma_commit(bar(C::ODone));
          }
          if (ok) {
            ok = wait(C::PReady + 1, steps1++ & 1u, kDevErrTimeoutMma, tiles);
            if (ok) {
              tc_fence_after();
              mma_pv(1, tiles == 1, vst);
              mma_commit(bar(C::KVEmpty + vst));
              mma_commit(bar(C::ODone + 1));
            }
          }
        } else {
          auto pv = [&](int j) -> bool {  // of tile j, group j mod 2
            const int g = j & 1;
            if (!v_ready(j, vst, vph) || !wait(C::PReady + g, (g ? steps1++ : steps0++) & 1u, kDevErrTimeoutMma, j))
              return false;
            tc_fence_after();
            mma_pv(g, j < 2, vst);
            mma_commit(bar(C::KVEmpty + vst));
            if (j + 2 >= tiles) mma_commit(bar(C::ODone + g));
            return true;
          };
          ok = wait(C::QFull + qs, (qs ? loads1++ : loads0++) & 1u, kDevErrTimeoutMma, (int)k);
          for (int j = 0; j < tiles && ok; ++j) {
            ok = wait(C::KVFull + kst, kph, kDevErrTimeoutMma, j);
            if (!ok) break;
            k_here(j);
            tc_fence_after();
            mma_s(j & 1, qs, kst);
            mma_commit(bar(C::KVEmpty + kst));
            if (j == tiles - 1) mma_commit(bar(C::QEmpty + qs));
            if (j > 0) ok = pv(j - 1);
            next(kst, kph);
            vst = kst;
            vph = kph;
            next(kst, kph);
          }
          if (ok) ok = pv(tiles - 1);
          qs ^= 1;
        }
      }
      ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
    }
    if (!ok && lane == 0) {
      // every MMA issued so far must finish reading shared memory and TMEM before exit
      mma_commit(bar(C::Drain));
      wait_phase(bar(C::Drain), 0, nullptr, p.timeout_ns, p.err, kDevErrTimeoutDrain, wtag(C::Drain, 0));
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ work, and its Q tiles
    // A piece of two row tiles has them in Q slots 0 and 1; pieces of one take the slots in turn, so
    // that the next one's Q lands while this one is at work.
    if (lane == 0) {
      const uint32_t q_bytes = (uint32_t)(C::PN * p.group * p.tq1 * 128);
      unsigned n_items = 0;
      StreamWalk walk;
      if constexpr (MODE == kStream) {
        walk.r = *run_of_cta;
      } else {
        n_items = p.counters[1];
      }
      uint32_t loads0 = 0, loads1 = 0;
      int qs = 0;
      bool more = true, ok = true;
      for (uint32_t k = 0; more; ++k) {
        // a piece is claimed when the producer is nearly through with the one before, not earlier:
        // claimed ahead, pieces would wait behind a long one while other CTAs run dry.  (A run's pieces are nobody
        // else's: trees take theirs as soon as there is room, 128 of 8 nodes over up to 1,000 keys 70.0 -> 68.5 us)
        if (k > 0 && !(TREE && MODE == kStream)) ok = wait_long(C::Want, (k - 1) & 1u, kDevErrTimeoutProducer, (int)k);
        if (!ok) break;
        SeqsItem it;
        if constexpr (MODE == kStream) {
          more = walk.next(p, it);
        } else {
          const unsigned e = atomicAdd(&p.counters[0], 1u);
          more = e < n_items;
          if (more) it = p.items[e];
        }
        if (!more) it.b = -1;
        const int slot = (int)(k & 1u);
        ok = wait_long(C::ItemEmpty + slot, ((k >> 1) & 1u) ^ 1u, kDevErrTimeoutProducer, (int)k);
        if (!ok) break;
        item_ring[slot] = it;
        mbar_arrive(bar(C::ItemFull + slot));
        if (!more || tiles_of(it) == 0) continue;
        const bool dual = it.nt > p.tq1;
        for (int t = 0; t < (dual ? 2 : 1) && ok; ++t) {
          const int qt = dual ? t : qs;
          const uint32_t before = qt ? loads1 : loads0;
          // the last S MMA on the slot's earlier contents
          if (before > 0) ok = wait_long(C::QEmpty + qt, (before - 1) & 1u, kDevErrTimeoutProducer, (int)k);
          if (!ok) break;
          mbar_expect_tx(bar(C::QFull + qt), q_bytes);
          for (int pn = 0; pn < C::PN; ++pn)
            tma_load_3d(base + C::offQ + qt * C::kTile + pn * kPanel, &maps.q, bar(C::QFull + qt), pn * 64, it.h * p.group,
                        it.qrow0 + t * p.tq1);
          if (qt) ++loads1; else ++loads0;
        }
        if (!ok) break;
        if (!dual) qs ^= 1;
      }
      if (!ok) {
        // every copy already issued lands before the CTA can exit
        if (loads0 > 0)
          wait_phase(bar(C::QFull), (loads0 - 1) & 1u, nullptr, p.timeout_ns, p.err, kDevErrTimeoutDrain, wtag(C::QFull, 0));
        if (loads1 > 0)
          wait_phase(bar(C::QFull + 1), (loads1 - 1) & 1u, nullptr, p.timeout_ns, p.err, kDevErrTimeoutDrain,
                     wtag(C::QFull + 1, 0));
      }
    }
  } else {
    // ------------------------------------------------------------ softmax groups
    // The tile loop needs most of the registers, so what only a piece's start and end use is taken
    // from the item ring again (its slot is given back at the end) or computed again.
    const int g = (warp - 4) >> 2;  // group
    const int wq = warp & 3;        // TMEM lane quarter of this warp
    const uint32_t tS = tmem + ((uint32_t)(wq * 32) << 16) + (uint32_t)(g * 128), tO = tS + 256u;
    auto token = [&](int row) -> int { return (int)((uint32_t)row * p.inv_group >> 16); };  // of a row of the tile
    uint32_t steps = 0, pieces0 = 0, pieces1 = 0, singles = 0;  // phases: S steps, O-done of both groups, Stat / EpiDone
    bool ok = true;
    for (uint32_t k = 0;; ++k) {
      const int slot = (int)(k & 1u);
      volatile const SeqsItem &it = item_ring[slot];
      if (lane == 0) ok = wait_long(C::ItemFull + slot, (k >> 1) & 1u, kDevErrTimeoutSoftmax, (int)k);
      ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
      __syncwarp();
      if (!ok || it.b < 0) break;
      const int key0 = it.key0, key1 = it.key1;
      const int tiles = key1 > key0 ? (key1 - key0 + 127) >> 7 : 0;
      const bool dual = it.nt > p.tq1;
      const int nsub = dual ? 2 * tiles : tiles;
      const int mine = (nsub - g + 1) >> 1;  // steps of this group
      float run, l[4] = {0.f, 0.f, 0.f, 0.f};
      {
        const int first_tok = dual ? g * p.tq1 : 0;
        const int left = min(p.tq1, it.nt - first_tok);  // tokens of this group's row tile
        const int tok0 = token(wq * 32), tok1 = token(wq * 32 + 31);  // tokens of the warp's rows
        const int tok = token(wq * 32 + opaque_laneid());
        const bool row_ok = tok < left;
        const int pos = it.pos0 + first_tok, kv = it.kv;
        int lo = 0, hi = 0;
        if (row_ok) seen_keys(pos + tok, kv, p.causal, p.window, lo, hi);
        // what every (used) row of the warp sees, for the tiles that need no mask
        int max_lo, min_hi, unused;
        seen_keys(pos + min(tok1, left - 1), kv, p.causal, p.window, max_lo, unused);
        seen_keys(pos + tok0, kv, p.causal, p.window, unused, min_hi);
        // a row that is no token's holds whatever its memory held: its max never asks for a rescale,
        // which the whole warp would take part in
        run = row_ok ? -INFINITY : INFINITY;
        TreeRow tree;
        if constexpr (TREE) {
          tree = tree_row(p.lens, p.mask, p.mask_words, p.mask_stride, it.b, it.kv, (int64_t)it.qrow0 + first_tok + tok, row_ok);
          min_hi = min(min_hi, tree.base);
        }
        if (tok0 >= left) min_hi = INT_MIN;  // no row of this warp is a token's
        int kb = key0 + (dual ? 0 : g * 128);
        const int kstep = dual ? 128 : 256;
        for (int i = 0; i < mine; ++i, kb += kstep) {
          ok = wait(C::SFull + g, (steps + (uint32_t)i) & 1u, kDevErrTimeoutSoftmax, i);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          if (min_hi != INT_MIN) {
            if constexpr (TREE) {
              if (kb + 128 > min_hi) mask_tree(tS, kb, hi, min_hi, tree.base, tree.bits, tree.words);
            } else {
              if (kb < max_lo || kb + 128 > min_hi) mask_rows(tS, kb, lo, hi, max_lo, min_hi);
            }
            softmax_tile<E, D, MODE == kLong ? 2 : 1>(tS, tO, p.alpha, i > 0, run, l);
            tmem_st_wait();
          }
          tc_fence_before();
          mbar_arrive(bar(C::PReady + g));
        }
      }
      steps += (uint32_t)mine;
      float lsum = (l[0] + l[1]) + (l[2] + l[3]);  // carries 2^(bias - run) (see p_bias)
      float2 *stat = reinterpret_cast<float2 *>(gbase + C::offStat) + wq * 32 + lane;
      if (!dual && g == 1) {
        // the other group joins the two results: it needs this group's max and sums, and O1 until
        // it says that it has read it
        *stat = make_float2(run, lsum);
        mbar_arrive(bar(C::Stat));
        ok = ok && wait(C::EpiDone, singles & 1u, kDevErrTimeoutSoftmax, (int)k);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      } else {
        float c0 = 1.f, c1 = 0.f;
        if (mine > 0) ok = ok && wait(C::ODone + g, (g ? pieces1 : pieces0) & 1u, kDevErrTimeoutSoftmax, (int)k);
        if (!dual) {
          // (group 1's arrival also says that it has seen O1 of its earlier pieces done, so that the
          // phase waited for next is the one after those)
          ok = ok && wait(C::Stat, singles & 1u, kDevErrTimeoutSoftmax, (int)k);
          if (nsub > 1) ok = ok && wait(C::ODone + 1, pieces1 & 1u, kDevErrTimeoutSoftmax, (int)k);
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (!dual) {
          const float2 o = *stat;
          const float m = fmaxf(run, o.x);
          c0 = run == -INFINITY ? 0.f : ex2(run - m);
          c1 = o.x == -INFINITY ? 0.f : ex2(o.x - m);
          lsum = lsum * c0 + o.y * c1;
          run = m;
        }
        const int first_tok = dual ? g * p.tq1 : 0;
        const int left = min(p.tq1, it.nt - first_tok);
        const int r = wq * 32 + opaque_laneid(), tok = token(r), hd = r - tok * p.group;
        const bool row_ok = tok < left;
        if (token(wq * 32) < left) {
          const int part = it.slot;
          const bool whole = part < 0;
          const float inv = !whole ? 1.f : (lsum == 0.f ? 0.f : 1.0f / lsum);  // no key seen: zeros, lse = -inf
          const float s0 = c0 * inv, s1 = c1 * inv;
          const int64_t qrow = (int64_t)it.qrow0 + first_tok + tok;
          const int head = it.h * p.group + hd;
          const int64_t slot_row = (int64_t)part * p.slot_rows + (first_tok + tok) * p.group + hd;
          const bool f32 = !whole || p.out_f32, wide = !whole || p.wide;  // (partial results are aligned)
          uint8_t *dst = whole ? reinterpret_cast<uint8_t *>(p.out) + (head * p.osH + qrow * p.osS) * (p.out_f32 ? 4 : 2)
                               : reinterpret_cast<uint8_t *>(p.part_o + slot_row * D);
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            float x[32];
            if (tiles > 0) {
              tmem_ld32(tO + c, o);
            } else {  // no key: O is an earlier piece's
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = 0u;
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(o[e]) * s0;
            if (!dual && nsub > 1) {
              tmem_ld32(tO + 128 + c, o);
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = fmaf(__uint_as_float(o[e]), s1, x[e]);
            }
            if (row_ok) store_row<E>(dst + c * (f32 ? 4 : 2), x, f32, wide);
          }
          if (row_ok) {
            // acc = sum 2^(z - run + bias): the bias leaves o as it is and comes off the log
            const float mx = run == -INFINITY ? run : run - p_bias<E>();
            if (!whole) p.part_ml[slot_row] = make_float2(mx, lsum);
            else if (p.lse)
              p.lse[head * p.T + qrow] = lsum == 0.f ? -INFINITY : 0.69314718055994531f * (mx + log2f(lsum));
          }
        }
        if (!dual) {
          tc_fence_before();
          mbar_arrive(bar(C::EpiDone));
        }
      }
      pieces0 += nsub > 0;
      pieces1 += nsub > 1;
      singles += dual ? 0 : 1;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(C::ItemEmpty + slot));
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

bool encode(CUtensorMap *map, const View &t, int rank, const cuuint64_t *dims, const cuuint64_t *strides, const cuuint32_t *box) {
  auto enc = get_encode();
  if (!enc) return false;
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  return enc(map, t.dtype == FM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank,
             const_cast<void *>(t.ptr), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Byte stride of a dimension; one of size 1 is never stepped and gets a well-formed value.
cuuint64_t step(int64_t s, int64_t n, int64_t other) { return (cuuint64_t)(n > 1 ? s : other) * 2; }

// q [1, Hq, T, D] as (D, Hq, T), box {64, group, tokens}.
bool encode_q(CUtensorMap *map, const View &t, int group, int tq1) {
  const cuuint64_t dims[3] = {(cuuint64_t)t.D, (cuuint64_t)t.H, (cuuint64_t)t.S};
  const cuuint64_t strides[2] = {step(t.sH, t.H, t.D), step(t.sS, t.S, t.H * t.D)};
  const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)tq1};
  return encode(map, t, 3, dims, strides, box);
}
// k or v [B, Hk, S, D] (pages, or one batch of packed rows) as (64, S, panels, Hk, B), a box of `rows`
// rows of all panels, or of one where a tile takes several boxes.
bool encode_kv(CUtensorMap *map, const View &t, int rows) {
  const cuuint64_t pn = (cuuint64_t)t.D / 64;
  const cuuint64_t dims[5] = {64, (cuuint64_t)t.S, pn, (cuuint64_t)t.H, (cuuint64_t)t.B};
  const cuuint64_t strides[4] = {step(t.sS, t.S, t.D), 128, step(t.sH, t.H, t.S * t.D), step(t.sB, t.B, t.H * t.S * t.D)};
  const cuuint32_t box[5] = {64, (cuuint32_t)rows, (cuuint32_t)(rows == 128 ? pn : 1), 1, 1};
  return encode(map, t, 5, dims, strides, box);
}
// Pages of fewer than 128 rows as (64, 8, panels, groups of 8 rows over all pages, Hk), a box of one
// page.  Wants pages that lie a whole number of groups apart.
bool encode_pages(CUtensorMap *map, const View &t) {
  const int64_t step8 = 8 * t.sS, per_page = t.B > 1 ? t.sB / step8 : t.S / 8;
  const cuuint64_t pn = (cuuint64_t)t.D / 64;
  const cuuint64_t dims[5] = {64, 8, pn, (cuuint64_t)((t.B - 1) * per_page + t.S / 8), (cuuint64_t)t.H};
  const cuuint64_t strides[4] = {(cuuint64_t)t.sS * 2, 128, (cuuint64_t)step8 * 2, step(t.sH, t.H, t.S * t.D)};
  const cuuint32_t box[5] = {64, 8, (cuuint32_t)pn, (cuuint32_t)(t.S / 8), 1};
  return encode(map, t, 5, dims, strides, box);
}
// Groups of 8 rows from one page to the next, 0: not a whole number (or too many to index).
int64_t page_groups(const View &t) {
  const int64_t step8 = 8 * t.sS;
  if (t.B > 1 && (t.sB % step8 || t.sB / step8 < t.S / 8)) return 0;
  const int64_t g = t.B > 1 ? t.sB / step8 : t.S / 8;
  return (t.B + 1) * g < ((int64_t)1 << 31) ? g : 0;
}

bool rows_aligned(const View &x, int64_t es, int64_t to) {
  auto ok = [&](int64_t s, int64_t n) { return n <= 1 || (s > 0 && (s * es) % to == 0 && s * es < ((int64_t)1 << 40)); };
  return x.sD == 1 && reinterpret_cast<uintptr_t>(x.ptr) % to == 0 && ok(x.sS, x.S) && ok(x.sH, x.H) && ok(x.sB, x.B);
}

template <typename E, int D, bool GROUPED, int MODE, bool TREE>
cudaError_t launch_typed(const Maps &maps, const Params &p, cudaStream_t st) {
  return launch_pdl(seqs_tc_kernel<E, D, GROUPED, MODE, TREE>, dim3((unsigned)current_device_sm_count()), dim3(kThreads),
                    Cfg<E, D, GROUPED>::kSmem, st, maps, p);
}
template <typename E, int D, bool GROUPED, int MODE, bool TREE>
cudaError_t allow_smem() {
  return cudaFuncSetAttribute(seqs_tc_kernel<E, D, GROUPED, MODE, TREE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              Cfg<E, D, GROUPED>::kSmem);
}
template <typename E, int D, bool TREE>
cudaError_t allow_smem_dim() {
  for (cudaError_t e : {allow_smem<E, D, true, kStream, TREE>(), allow_smem<E, D, true, kList, TREE>(),
                        allow_smem<E, D, false, kStream, TREE>(), allow_smem<E, D, false, kList, TREE>(),
                        allow_smem<E, D, false, D == 64 && !TREE ? kLong : kList, TREE>()})
    if (e != cudaSuccess) return e;
  return cudaSuccess;
}
template <typename E, int D, bool TREE>
cudaError_t launch_dim(const Maps &maps, const Params &p, bool grouped, int mode, cudaStream_t st) {
  if (grouped) {
    if (mode == kStream) return launch_typed<E, D, true, kStream, TREE>(maps, p, st);
    return launch_typed<E, D, true, kList, TREE>(maps, p, st);
  }
  if (mode == kStream) return launch_typed<E, D, false, kStream, TREE>(maps, p, st);
  if constexpr (D == 64 && !TREE)
    if (mode == kLong) return launch_typed<E, D, false, kLong, TREE>(maps, p, st);
  return launch_typed<E, D, false, kList, TREE>(maps, p, st);
}

template <bool TREE>
cudaError_t prepare_tc() {
  for (cudaError_t e : {allow_smem_dim<__nv_bfloat16, 128, TREE>(), allow_smem_dim<__nv_bfloat16, 64, TREE>(),
                        allow_smem_dim<__half, 128, TREE>(), allow_smem_dim<__half, 64, TREE>()})
    if (e != cudaSuccess) return e;
  return cudaSuccess;
}

template <bool TREE>
cudaError_t launch_tc(const SeqsArgs &a, const SeqsGeom &g, const SeqsSpace &s, cudaStream_t st) {
  uint8_t *ws = static_cast<uint8_t *>(a.ws);
  Maps maps;
  memset(&maps, 0, sizeof maps);
  Params p;
  p.group = g.group;
  p.tq1 = g.tq / 2;
  p.inv_group = (65536u + (uint32_t)g.group - 1u) / (uint32_t)g.group;
  p.wide = rows_aligned(a.o, a.o.dtype == FM_F32 ? 4 : 2, 32);
  p.box_rows = a.paged && a.k.S < 128 ? (int)a.k.S : 128;
  const int64_t groups = p.box_rows < 128 ? page_groups(a.k) : 0;
  const bool grouped = groups > 0 && groups == page_groups(a.v);
  p.page_groups = (int)groups;
  if (!encode_q(&maps.q, a.q, p.group, p.tq1) ||
      !(grouped ? encode_pages(&maps.k, a.k) && encode_pages(&maps.v, a.v)
                  : encode_kv(&maps.k, a.k, p.box_rows) && encode_kv(&maps.v, a.v, p.box_rows)))
    return cudaErrorNotSupported;
  p.causal = a.causal;
  p.window = a.window;
  p.alpha = a.alpha;
  p.paged = a.paged;
  p.ps = a.paged ? (int)a.k.S : 1;
  p.num_pages = a.paged ? (int)a.k.B : 0;
  p.table = a.table;
  p.table_stride = a.table_stride;
  p.counters = reinterpret_cast<unsigned int *>(ws + s.counters);
  p.items = reinterpret_cast<const SeqsItem *>(ws + s.items);
  p.merges = reinterpret_cast<SeqsMerge *>(ws + s.merges);
  p.lens = seqs_lens(a);
  p.n = (int)a.n;
  p.Hk = (int)a.k.H;
  p.part_o = reinterpret_cast<float *>(ws + s.part_o);
  p.part_ml = reinterpret_cast<float2 *>(ws + s.part_ml);
  p.slot_rows = g.slot_rows;
  p.out = const_cast<void *>(a.o.ptr);
  p.out_f32 = a.o.dtype == FM_F32;
  p.osH = a.o.sH;
  p.osS = a.o.sS;
  p.lse = a.lse;
  p.T = a.q.S;
  p.mask = a.mask;
  p.mask_words = (int)a.mask_words;
  p.mask_stride = a.mask_stride;
  p.err = a.err;
  p.timeout_ns = a.timeout_ns;
  // packed prompts of 4,096 queries and more on average (of the arrays' rows), D = 64 (see softmax_tile)
  const int mode = g.stream ? kStream : (a.q.D == 64 && !a.paged && a.q.S >= 4096 * a.n ? kLong : kList);
  if (a.q.dtype == FM_BF16)
    return a.q.D == 128 ? launch_dim<__nv_bfloat16, 128, TREE>(maps, p, grouped, mode, st)
                        : launch_dim<__nv_bfloat16, 64, TREE>(maps, p, grouped, mode, st);
  return a.q.D == 128 ? launch_dim<__half, 128, TREE>(maps, p, grouped, mode, st)
                      : launch_dim<__half, 64, TREE>(maps, p, grouped, mode, st);
}

}  // namespace
}  // namespace fm
