// fm_seqs_simt.cuh -- attention over requests of different lengths on the CUDA cores.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(alpha q_i.k_j - r_i),  r_i the running row max
// over the keys j that token i sees (causal, window, the request's length).  Serves fp32 inputs
// (exact fp32 arithmetic) and the 16-bit layouts that the tensor-core kernel does not take
// (strides that a tensor map cannot describe, page sizes that do not fit its tiles).
//
// One CTA takes pieces of work from the list: 64 rows (tokens x query heads of one key head, so
// that the heads that share a key head read it once) against 64-key tiles.  256 threads as 16 x
// 16: a thread holds 4 rows x 4 keys of the scores and 4 rows x D/16 columns of o in registers,
// and reads its operands from shared memory as 16-byte words: 12 (scores) to 20 (output) shared
// wavefronts for 64 to 128 FMAs a thread, so that the FMA pipe and not shared memory bounds the
// long cases.  K and V of a tile share one buffer, so that two CTAs fit an SM and one's loads run
// beside the other's arithmetic.  fp32, one prompt of 16,384, D = 128: 36 TFLOP/s (of 75); four of 2,048
// at D = 64: 25.
// Units of at most 16 rows have a kernel of their own (seqs_few_kernel).
// TREE (fm_attn_tree): of its request's new tokens a row sees those that its mask row names.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "fm_seqs.cuh"

namespace fm {
namespace {

constexpr int kR = 64, kK = 64, kT = 256;  // rows, keys and threads of a CTA

struct SimtArgs {
  View q, k, v, o;
  int paged;
  const int32_t *table;
  int64_t table_stride;
  int ps, num_pages;
  float alpha;
  int causal, window, group, slot_rows;
  int64_t T;
  float *lse;
  unsigned int *counters;
  const SeqsItem *items;
  float *part_o;
  float2 *part_ml;
  unsigned int *err;
  SeqsLens lens;         // TREE, as the rest: rows of mask_words words, mask_stride apart
  const uint32_t *mask;
  int mask_words;
  int64_t mask_stride;
};
__device__ __forceinline__ TreeRow tree_row(const SimtArgs &a, const SeqsItem &it, int r, bool ok) {
  return tree_row(a.lens, a.mask, a.mask_words, a.mask_stride, it.b, it.kv, (int64_t)it.qrow0 + r / a.group, ok);
}

__device__ __forceinline__ float as_f32(float x) { return x; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float as_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ void put(float *p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void put(__half *p, float x) { *p = __float2half_rn(x); }

// Four consecutive elements of a row as fp32; VEC: unit stride and aligned, one load.
template <typename E>
__device__ __forceinline__ float4 load4(const E *p, int64_t sD, bool vec) {
  if (vec) {
    if constexpr (sizeof(E) == 4) return *reinterpret_cast<const float4 *>(p);
    else {
      const uint2 u = *reinterpret_cast<const uint2 *>(p);
      const E *e = reinterpret_cast<const E *>(&u);
      return make_float4(as_f32(e[0]), as_f32(e[1]), as_f32(e[2]), as_f32(e[3]));
    }
  }
  return make_float4(as_f32(p[0]), as_f32(p[sD]), as_f32(p[2 * sD]), as_f32(p[3 * sD]));
}

// The row of key j of the item's request in K or V (nullptr: an entry outside the cache, whose
// keys and values read as zeros).
template <typename E>
__device__ __forceinline__ const E *key_row(const SimtArgs &a, const View &x, const SeqsItem &it, int j) {
  const E *base = reinterpret_cast<const E *>(x.ptr) + it.h * x.sH;
  if (!a.paged) return base + (int64_t)(it.krow0 + j) * x.sS;
  const int pg = a.table[it.b * a.table_stride + j / a.ps];
  if (pg < 0 || pg >= a.num_pages) {
    report_bad_page(a.err, it.b, j / a.ps, pg);
    return nullptr;
  }
  return base + pg * x.sB + (int64_t)(j % a.ps) * x.sS;
}

template <typename E, typename O, int D, bool TREE>
__global__ void __launch_bounds__(kT, 2) seqs_simt_kernel(const SimtArgs a, const bool vec) {
  constexpr int SQ = D + 4, SP = kK + 4;  // padded rows: 16-byte reads of 8 rows cover the 32 banks
  constexpr int CPT = D / 16;             // output columns of a thread
  extern __shared__ __align__(16) float smem[];
  float *Qs = smem, *KVs = Qs + kR * SQ, *Ps = KVs + kK * SQ;
  __shared__ int next_s;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const unsigned n_items = a.counters[1];
  for (;;) {
    if (tid == 0) next_s = (int)atomicAdd(&a.counters[0], 1u);
    __syncthreads();
    const unsigned idx = (unsigned)next_s;
    if (idx >= n_items) return;
    const SeqsItem it = a.items[idx];
    const int rows = it.nt * a.group;
    const int seen0 = a.window > 0 ? max(0, it.pos0 - a.window + 1) : 0;  // earlier keys no token of the unit sees
    const E *qp = reinterpret_cast<const E *>(a.q.ptr) + (int64_t)it.h * a.group * a.q.sH + (int64_t)it.qrow0 * a.q.sS;
    for (int i = tid; i < kR * (D / 4); i += kT) {
      const int r = i / (D / 4), d = (i % (D / 4)) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) x = load4(qp + (r % a.group) * a.q.sH + (r / a.group) * a.q.sS + d * a.q.sD, a.q.sD, vec);
      *reinterpret_cast<float4 *>(Qs + r * SQ + d) = x;
    }
    int lo[4], hi[4];
    TreeRow tree[4];
    float run[4], l[4], acc[4][CPT];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i;
      lo[i] = hi[i] = 0;
      if (r < rows) seen_keys(it.pos0 + r / a.group, it.kv, a.causal, a.window, lo[i], hi[i]);
      hi[i] = min(hi[i], it.key1);
      if constexpr (TREE) tree[i] = tree_row(a, it, r, r < rows);
      run[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < CPT; ++c) acc[i][c] = 0.f;
    }
    for (int j0 = it.key0; j0 < it.key1; j0 += kK) {
      __syncthreads();  // Q is stored; the last tile's V and P have been read
      for (int i = tid; i < kK * (D / 4); i += kT) {
        const int j = i / (D / 4), d = (i % (D / 4)) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j0 + j >= seen0 && j0 + j < it.key1) {
          const E *p = key_row<E>(a, a.k, it, j0 + j);
          if (p) x = load4(p + d * a.k.sD, a.k.sD, vec);
        }
        *reinterpret_cast<float4 *>(KVs + j * SQ + d) = x;
      }
      __syncthreads();
      float s[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 qv[4], kv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) qv[i] = *reinterpret_cast<const float4 *>(Qs + (ty * 4 + i) * SQ + d);
#pragma unroll
        for (int j = 0; j < 4; ++j) kv[j] = *reinterpret_cast<const float4 *>(KVs + (tx + 16 * j) * SQ + d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[i][j] = fmaf(qv[i].x, kv[j].x, s[i][j]);
            s[i][j] = fmaf(qv[i].y, kv[j].y, s[i][j]);
            s[i][j] = fmaf(qv[i].z, kv[j].z, s[i][j]);
            s[i][j] = fmaf(qv[i].w, kv[j].w, s[i][j]);
          }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = j0 + tx + 16 * j;
          bool seen = key >= lo[i] && key < hi[i];
          if constexpr (TREE) seen = seen && tree_sees(tree[i], key);
          s[i][j] = seen ? s[i][j] * a.alpha : -INFINITY;
          mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float nr = fmaxf(run[i], mx);
        const float shift = nr == -INFINITY ? 0.f : nr;  // no key seen so far: every p below is 2^-inf = 0
        const float c = exp2f(run[i] - shift);
        float ps = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = exp2f(s[i][j] - shift);
          ps += s[i][j];
          Ps[(ty * 4 + i) * SP + tx + 16 * j] = s[i][j];
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, d);
        l[i] = fmaf(l[i], c, ps);
        run[i] = nr;
#pragma unroll
        for (int cc = 0; cc < CPT; ++cc) acc[i][cc] *= c;
      }
      __syncthreads();  // K has been read, P is stored
      for (int i = tid; i < kK * (D / 4); i += kT) {
        const int j = i / (D / 4), d = (i % (D / 4)) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (j0 + j >= seen0 && j0 + j < it.key1) {
          const E *p = key_row<E>(a, a.v, it, j0 + j);
          if (p) x = load4(p + d * a.v.sD, a.v.sD, vec);
        }
        *reinterpret_cast<float4 *>(KVs + j * SQ + d) = x;
      }
      __syncthreads();
#pragma unroll 2
      for (int j = 0; j < kK; j += 4) {
        float4 pv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) pv[i] = *reinterpret_cast<const float4 *>(Ps + (ty * 4 + i) * SP + j);
#pragma unroll
        for (int jj = 0; jj < 4; ++jj)
#pragma unroll
          for (int c = 0; c < CPT; c += 4) {
            const float4 vv = *reinterpret_cast<const float4 *>(KVs + (j + jj) * SQ + tx * 4 + c * 16);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float p = jj == 0 ? pv[i].x : jj == 1 ? pv[i].y : jj == 2 ? pv[i].z : pv[i].w;
              acc[i][c] = fmaf(p, vv.x, acc[i][c]);
              acc[i][c + 1] = fmaf(p, vv.y, acc[i][c + 1]);
              acc[i][c + 2] = fmaf(p, vv.z, acc[i][c + 2]);
              acc[i][c + 3] = fmaf(p, vv.w, acc[i][c + 3]);
            }
          }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i;
      if (r >= rows) continue;
      if (it.slot >= 0) {
        const int64_t at = (int64_t)it.slot * a.slot_rows + r;
        for (int c = 0; c < CPT; c += 4)
          *reinterpret_cast<float4 *>(a.part_o + at * D + tx * 4 + c * 16) =
              make_float4(acc[i][c], acc[i][c + 1], acc[i][c + 2], acc[i][c + 3]);
        if (tx == 0) a.part_ml[at] = make_float2(run[i], l[i]);
        continue;
      }
      const float inv = l[i] == 0.f ? 0.f : 1.0f / l[i];  // a row that sees no key: zeros, lse = -inf
      const int head = it.h * a.group + r % a.group;
      const int64_t tok = it.qrow0 + r / a.group;
      O *dst = reinterpret_cast<O *>(const_cast<void *>(a.o.ptr)) + head * a.o.sH + tok * a.o.sS;
#pragma unroll
      for (int c = 0; c < CPT; ++c)
        put(dst + (int64_t)(tx * 4 + (c & 3) + (c >> 2) * 64) * a.o.sD, acc[i][c] * inv);
      if (a.lse && tx == 0)
        a.lse[head * a.T + tok] = l[i] == 0.f ? -INFINITY : 0.69314718055994531f * (run[i] + log2f(l[i]));
    }
    __syncthreads();  // next_s and Q are replaced
  }
}

// ---------------------------------------------------------------- few rows: decoding
// Where a unit has at most R = 8 or 16 rows, a tile of 64 leaves most of the arithmetic and of the
// shared-memory traffic to rows that are none.  Here a warp takes 32 keys at a time by itself, K and
// V going from memory to registers: 8 lanes hold a key (4 keys a step), the partial dot products of 8
// rows are summed over those lanes by 7 exchanges that leave each lane one row's score, and for O a
// lane holds 4 columns of all rows.  The warps' sums are joined at the end of a piece, in order.
// Bound by the latency of its loads and by issue (about 100 instructions a key and 8 rows); fp32, 64
// requests of up to 8,192 keys, 8 key heads, D = 128: 379 us with 8 rows (3.9 TB/s), 756 with 16,
// 1,911 by the kernel above; bf16 on pages of 24 keys 473.  16 value rows in flight: 397 -> 379 us;
// values asked for ahead: 819 -> 756 (16 rows), 578 -> 473 (bf16), and nothing for 8 rows of fp32;
// keys asked for ahead too, more CTAs with fewer registers, or 4 keys at a time are slower (469,
// 544, 437).
constexpr int kWarps = 8, kBlock = 32;  // warps of a CTA, keys of a warp's step

template <int D, int R>
struct Few {
  static constexpr int KD = D / 32;          // 4-column groups of a key that a lane holds
  static constexpr int VL = D / 4, KV = 32 / VL;  // lanes of a value row, value rows of a step
  static constexpr int offP = R * D, offO = offP + kWarps * kBlock * R, offML = offO + kWarps * R * D;
  static constexpr int bytes = (offML + kWarps * R * 2) * 4;
};

template <typename E, typename O, int D, int R, bool TREE>
__global__ void __launch_bounds__(32 * kWarps, 2) seqs_few_kernel(const SimtArgs a, const bool vec) {
  using F = Few<D, R>;
  constexpr int KD = F::KD, RB = R / 8, W = R == 8 ? 2 : 1;  // W: steps of 4 keys at a time
  extern __shared__ __align__(16) float smem[];
  __shared__ int next_s;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, kg = lane >> 3, row8 = lane & 7;
  float *Qs = smem, *Ps = smem + F::offP + warp * kBlock * R, *Os = smem + F::offO;
  float2 *ML = reinterpret_cast<float2 *>(smem + F::offML);
  const unsigned n_items = a.counters[1];
  for (;;) {
    if (tid == 0) next_s = (int)atomicAdd(&a.counters[0], 1u);
    __syncthreads();
    const unsigned idx = (unsigned)next_s;
    if (idx >= n_items) return;
    const SeqsItem it = a.items[idx];
    const int rows = it.nt * a.group;
    const int seen0 = a.window > 0 ? max(0, it.pos0 - a.window + 1) : 0;  // earlier keys no token of the unit sees
    const E *qp = reinterpret_cast<const E *>(a.q.ptr) + (int64_t)it.h * a.group * a.q.sH + (int64_t)it.qrow0 * a.q.sS;
    for (int i = tid; i < R * (D / 4); i += 32 * kWarps) {
      const int r = i / (D / 4), d = (i % (D / 4)) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) x = load4(qp + (r % a.group) * a.q.sH + (r / a.group) * a.q.sS + d * a.q.sD, a.q.sD, vec);
      *reinterpret_cast<float4 *>(Qs + r * D + d) = x;
    }
    int lo[RB], hi[RB];  // keys seen by this lane's rows
    TreeRow tree[RB];
    float run[RB], l[RB], acc[R][4];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      const int r = b * 8 + row8;
      lo[b] = hi[b] = 0;
      if (r < rows) seen_keys(it.pos0 + r / a.group, it.kv, a.causal, a.window, lo[b], hi[b]);
      hi[b] = min(hi[b], it.key1);
      if constexpr (TREE) tree[b] = tree_row(a, it, r, r < rows);
      run[b] = -INFINITY;
      l[b] = 0.f;
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[r][e] = 0.f;
    __syncthreads();  // Q is stored
    // where key j0 + lane lies: page (packed: 0) and row, page -1: reads as zeros
    auto place = [&](int j0, int &page, int &row) {
      const int j = j0 + lane;
      page = -1;
      row = 0;
      if (j < seen0 || j >= it.key1) return;
      if (!a.paged) {
        page = 0;
        row = it.krow0 + j;
        return;
      }
      const int at = j / a.ps;
      row = j - at * a.ps;
      page = a.table[it.b * a.table_stride + at];
      if (page < 0 || page >= a.num_pages) {
        report_bad_page(a.err, it.b, at, page);
        page = -1;
      }
    };
    const E *kb = reinterpret_cast<const E *>(a.k.ptr) + it.h * a.k.sH + row8 * 4 * a.k.sD;
    const E *vb = reinterpret_cast<const E *>(a.v.ptr) + it.h * a.v.sH + (lane % F::VL) * 4 * a.v.sD;
    int page, row;
    place(it.key0 + warp * kBlock, page, row);
    for (int j0 = it.key0 + warp * kBlock; j0 < it.key1; j0 += kWarps * kBlock) {
      int page_next, row_next;
      place(j0 + kWarps * kBlock, page_next, row_next);
      // the values on their way to L2 while the scores are computed (where fewer of their loads fit the
      // registers, or bring half the bytes)
      if constexpr (R == 16 || sizeof(E) == 2) {
        if (vec && page >= 0) {
          const E *vr = reinterpret_cast<const E *>(a.v.ptr) + it.h * a.v.sH + page * a.v.sB + row * a.v.sS;
#pragma unroll
          for (int d = 0; d < D; d += 128 / (int)sizeof(E)) asm volatile("prefetch.global.L2 [%0];" ::"l"(vr + d));
        }
      }
      // 1. scores of 32 keys
      float mx[RB];
#pragma unroll
      for (int b = 0; b < RB; ++b) mx[b] = -INFINITY;
#pragma unroll 1
      for (int u = 0; u < kBlock / 4; u += W) {
        float4 k[W][KD];
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const int pg = __shfl_sync(0xffffffffu, page, (u + w) * 4 + kg), rw = __shfl_sync(0xffffffffu, row, (u + w) * 4 + kg);
          const E *p = kb + pg * a.k.sB + rw * a.k.sS;
#pragma unroll
          for (int i = 0; i < KD; ++i)
            k[w][i] = pg >= 0 ? load4(p + i * 32 * a.k.sD, a.k.sD, vec) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          float s[W][8];
#pragma unroll
          for (int r = 0; r < 8; ++r) {
#pragma unroll
            for (int w = 0; w < W; ++w) s[w][r] = 0.f;
#pragma unroll
            for (int i = 0; i < KD; ++i) {
              const float4 q = *reinterpret_cast<const float4 *>(Qs + (b * 8 + r) * D + i * 32 + row8 * 4);
#pragma unroll
              for (int w = 0; w < W; ++w) {
                s[w][r] = fmaf(q.x, k[w][i].x, s[w][r]);
                s[w][r] = fmaf(q.y, k[w][i].y, s[w][r]);
                s[w][r] = fmaf(q.z, k[w][i].z, s[w][r]);
                s[w][r] = fmaf(q.w, k[w][i].w, s[w][r]);
              }
            }
          }
#pragma unroll
          for (int w = 0; w < W; ++w) {
            // the 8 lanes' sums: each exchange halves the rows that a lane goes on with
#pragma unroll
            for (int half = 4; half > 0; half >>= 1) {
              const bool up = (lane & half) != 0;
#pragma unroll
              for (int r = 0; r < half; ++r) {
                const float give = up ? s[w][r] : s[w][r + half], keep = up ? s[w][r + half] : s[w][r];
                s[w][r] = keep + __shfl_xor_sync(0xffffffffu, give, half);
              }
            }
            const int j = (u + w) * 4 + kg, key = j0 + j;
            bool seen = key >= lo[b] && key < hi[b];
            if constexpr (TREE) seen = seen && tree_sees(tree[b], key);
            const float x = seen ? s[w][0] * a.alpha : -INFINITY;
            mx[b] = fmaxf(mx[b], x);
            Ps[j * R + b * 8 + row8] = x;
          }
        }
      }
      // 2. the rows' max and weights; a lane has its row's scores of every 4th key
      float c[RB];
      bool moved = false;
#pragma unroll
      for (int b = 0; b < RB; ++b) {
        mx[b] = fmaxf(mx[b], __shfl_xor_sync(0xffffffffu, mx[b], 8));
        mx[b] = fmaxf(mx[b], __shfl_xor_sync(0xffffffffu, mx[b], 16));
        const float nr = fmaxf(run[b], mx[b]);
        const float shift = nr == -INFINITY ? 0.f : nr;  // no key seen so far: every p below is 2^-inf = 0
        c[b] = exp2f(run[b] - shift);
        moved |= nr != run[b];
        run[b] = nr;
        float ps = 0.f;
#pragma unroll
        for (int u = 0; u < kBlock / 4; ++u) {
          float *at = Ps + (u * 4 + kg) * R + b * 8 + row8;
          const float p = exp2f(*at - shift);
          ps += p;
          *at = p;
        }
        l[b] = fmaf(l[b], c[b], ps);
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float cr = __shfl_sync(0xffffffffu, c[r / 8], r & 7);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[r][e] *= cr;
        }
      }
      __syncwarp();  // the weights are stored
      // 3. O += P V
#pragma unroll R == 8 ? 16 : 8
      for (int u = 0; u < kBlock; u += F::KV) {
        const int j = u + lane / F::VL;
        const int pg = __shfl_sync(0xffffffffu, page, j), rw = __shfl_sync(0xffffffffu, row, j);
        const float4 v = pg >= 0 ? load4(vb + pg * a.v.sB + rw * a.v.sS, a.v.sD, vec) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int r = 0; r < R; r += 4) {
          const float4 p = *reinterpret_cast<const float4 *>(Ps + j * R + r);
          const float pr[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc[r + e][0] = fmaf(pr[e], v.x, acc[r + e][0]);
            acc[r + e][1] = fmaf(pr[e], v.y, acc[r + e][1]);
            acc[r + e][2] = fmaf(pr[e], v.z, acc[r + e][2]);
            acc[r + e][3] = fmaf(pr[e], v.w, acc[r + e][3]);
          }
        }
      }
      __syncwarp();  // the weights have been read
      page = page_next;
      row = row_next;
    }
    // the warps' results: o = sum_w 2^(m_w - M) o_w, and the sums likewise
#pragma unroll
    for (int b = 0; b < RB; ++b) {
      l[b] += __shfl_xor_sync(0xffffffffu, l[b], 8);
      l[b] += __shfl_xor_sync(0xffffffffu, l[b], 16);
      if (lane < 8) ML[warp * R + b * 8 + lane] = make_float2(run[b], l[b]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float4 x = make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
      if constexpr (F::KV == 2) {
        x.x += __shfl_xor_sync(0xffffffffu, x.x, 16);
        x.y += __shfl_xor_sync(0xffffffffu, x.y, 16);
        x.z += __shfl_xor_sync(0xffffffffu, x.z, 16);
        x.w += __shfl_xor_sync(0xffffffffu, x.w, 16);
      }
      if (lane < F::VL) *reinterpret_cast<float4 *>(Os + (warp * R + r) * D + lane * 4) = x;
    }
    __syncthreads();
    for (int i = tid; i < rows * (D / 4); i += 32 * kWarps) {
      const int r = i / (D / 4), d = (i % (D / 4)) * 4;
      float M = -INFINITY, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ML[w * R + r].x);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 ml = ML[w * R + r];
        const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
        const float4 y = *reinterpret_cast<const float4 *>(Os + (w * R + r) * D + d);
        sum = fmaf(ml.y, f, sum);
        x.x = fmaf(y.x, f, x.x);
        x.y = fmaf(y.y, f, x.y);
        x.z = fmaf(y.z, f, x.z);
        x.w = fmaf(y.w, f, x.w);
      }
      if (it.slot >= 0) {
        const int64_t at = (int64_t)it.slot * a.slot_rows + r;
        *reinterpret_cast<float4 *>(a.part_o + at * D + d) = x;
        if (d == 0) a.part_ml[at] = make_float2(M, sum);
        continue;
      }
      const float inv = sum == 0.f ? 0.f : 1.0f / sum;  // a row that sees no key: zeros, lse = -inf
      const int head = it.h * a.group + r % a.group;
      const int64_t tok = it.qrow0 + r / a.group;
      O *dst = reinterpret_cast<O *>(const_cast<void *>(a.o.ptr)) + head * a.o.sH + tok * a.o.sS + d * a.o.sD;
      put(dst, x.x * inv);
      put(dst + a.o.sD, x.y * inv);
      put(dst + 2 * a.o.sD, x.z * inv);
      put(dst + 3 * a.o.sD, x.w * inv);
      if (a.lse && d == 0)
        a.lse[head * a.T + tok] = sum == 0.f ? -INFINITY : 0.69314718055994531f * (M + log2f(sum));
    }
    // (next_s, Q and the warps' results are replaced after the barrier at the loop's start)
  }
}

template <int D>
constexpr int smem_bytes = (kR * (D + 4) + kK * (D + 4) + kR * (kK + 4)) * 4;

template <typename E, typename O, int D, bool TREE>
cudaError_t launch_typed(const SimtArgs &p, const SeqsGeom &g, bool vec, cudaStream_t st) {
  const dim3 grid((unsigned)current_device_sm_count() * 2);
  const int rows = g.tq * g.group;
  if (rows <= 8) return launch_pdl(seqs_few_kernel<E, O, D, 8, TREE>, grid, dim3(32 * kWarps), Few<D, 8>::bytes, st, p, vec);
  if (rows <= 16) return launch_pdl(seqs_few_kernel<E, O, D, 16, TREE>, grid, dim3(32 * kWarps), Few<D, 16>::bytes, st, p, vec);
  return launch_pdl(seqs_simt_kernel<E, O, D, TREE>, grid, dim3(kT), smem_bytes<D>, st, p, vec);
}
template <typename E, typename O, int D, bool TREE>
cudaError_t allow_smem_of() {
  const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  for (cudaError_t e : {cudaFuncSetAttribute(seqs_simt_kernel<E, O, D, TREE>, attr, smem_bytes<D>),
                        cudaFuncSetAttribute(seqs_few_kernel<E, O, D, 8, TREE>, attr, Few<D, 8>::bytes),
                        cudaFuncSetAttribute(seqs_few_kernel<E, O, D, 16, TREE>, attr, Few<D, 16>::bytes)})
    if (e != cudaSuccess) return e;
  return cudaSuccess;
}
template <typename E, typename O, bool TREE>
cudaError_t allow_smem() {
  const cudaError_t e = allow_smem_of<E, O, 128, TREE>();
  return e == cudaSuccess ? allow_smem_of<E, O, 64, TREE>() : e;
}

template <typename E, bool TREE>
cudaError_t launch_elem(const SimtArgs &p, const SeqsGeom &g, bool vec, cudaStream_t st) {
  if (p.o.dtype == FM_F32)
    return p.o.D == 128 ? launch_typed<E, float, 128, TREE>(p, g, vec, st) : launch_typed<E, float, 64, TREE>(p, g, vec, st);
  return p.o.D == 128 ? launch_typed<E, E, 128, TREE>(p, g, vec, st) : launch_typed<E, E, 64, TREE>(p, g, vec, st);
}

bool quads(const View &x, int64_t es) {
  auto ok = [&](int64_t s, int64_t n) { return n <= 1 || s % 4 == 0; };
  return x.sD == 1 && reinterpret_cast<uintptr_t>(x.ptr) % (4 * es) == 0 && ok(x.sS, x.S) && ok(x.sH, x.H) && ok(x.sB, x.B);
}

template <bool TREE>
cudaError_t prepare_simt() {
  for (cudaError_t e : {allow_smem<float, float, TREE>(), allow_smem<__nv_bfloat16, float, TREE>(),
                        allow_smem<__nv_bfloat16, __nv_bfloat16, TREE>(), allow_smem<__half, float, TREE>(),
                        allow_smem<__half, __half, TREE>()})
    if (e != cudaSuccess) return e;
  return cudaSuccess;
}

template <bool TREE>
cudaError_t launch_simt(const SeqsArgs &a, const SeqsGeom &g, const SeqsSpace &s, cudaStream_t st) {
  uint8_t *ws = static_cast<uint8_t *>(a.ws);
  SimtArgs p;
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.o = a.o;
  p.paged = a.paged;
  p.table = a.table;
  p.table_stride = a.table_stride;
  p.ps = a.paged ? (int)a.k.S : 1;
  p.num_pages = a.paged ? (int)a.k.B : 0;
  p.alpha = a.alpha;
  p.causal = a.causal;
  p.window = a.window;
  p.group = g.group;
  p.slot_rows = g.slot_rows;
  p.T = a.q.S;
  p.lse = a.lse;
  p.counters = reinterpret_cast<unsigned int *>(ws + s.counters);
  p.items = reinterpret_cast<const SeqsItem *>(ws + s.items);
  p.part_o = reinterpret_cast<float *>(ws + s.part_o);
  p.part_ml = reinterpret_cast<float2 *>(ws + s.part_ml);
  p.err = a.err;
  p.lens = seqs_lens(a);
  p.mask = a.mask;
  p.mask_words = (int)a.mask_words;
  p.mask_stride = a.mask_stride;
  const int64_t es = a.q.dtype == FM_F32 ? 4 : 2;
  const bool vec = quads(a.q, es) && quads(a.k, es) && quads(a.v, es);
  if (a.q.dtype == FM_F32) return launch_elem<float, TREE>(p, g, vec, st);
  if (a.q.dtype == FM_BF16) return launch_elem<__nv_bfloat16, TREE>(p, g, vec, st);
  return launch_elem<__half, TREE>(p, g, vec, st);
}

}  // namespace
}  // namespace fm
