// fm_seqs_simt.cu -- attention over requests of different lengths on the CUDA cores.
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
// beside the other's arithmetic.
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
};

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

template <typename E, typename O, int D>
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
    float run[4], l[4], acc[4][CPT];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i;
      lo[i] = hi[i] = 0;
      if (r < rows) seen_keys(it.pos0 + r / a.group, it.kv, a.causal, a.window, lo[i], hi[i]);
      hi[i] = min(hi[i], it.key1);
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
          s[i][j] = (key >= lo[i] && key < hi[i]) ? s[i][j] * a.alpha : -INFINITY;
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

template <int D>
constexpr int smem_bytes = (kR * (D + 4) + kK * (D + 4) + kR * (kK + 4)) * 4;

template <typename E, typename O, int D>
cudaError_t launch_typed(const SimtArgs &p, bool vec, cudaStream_t st) {
  return launch_pdl(seqs_simt_kernel<E, O, D>, dim3((unsigned)current_device_sm_count() * 2), dim3(kT), smem_bytes<D>, st, p,
                    vec);
}
template <typename E, typename O>
cudaError_t allow_smem() {
  const cudaError_t e =
      cudaFuncSetAttribute(seqs_simt_kernel<E, O, 128>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<128>);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(seqs_simt_kernel<E, O, 64>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes<64>);
}

template <typename E>
cudaError_t launch_elem(const SimtArgs &p, bool vec, cudaStream_t st) {
  if (p.o.dtype == FM_F32)
    return p.o.D == 128 ? launch_typed<E, float, 128>(p, vec, st) : launch_typed<E, float, 64>(p, vec, st);
  return p.o.D == 128 ? launch_typed<E, E, 128>(p, vec, st) : launch_typed<E, E, 64>(p, vec, st);
}

bool quads(const View &x, int64_t es) {
  auto ok = [&](int64_t s, int64_t n) { return n <= 1 || s % 4 == 0; };
  return x.sD == 1 && reinterpret_cast<uintptr_t>(x.ptr) % (4 * es) == 0 && ok(x.sS, x.S) && ok(x.sH, x.H) && ok(x.sB, x.B);
}

}  // namespace

cudaError_t seqs_simt_prepare() {
  for (cudaError_t e : {allow_smem<float, float>(), allow_smem<__nv_bfloat16, float>(), allow_smem<__nv_bfloat16, __nv_bfloat16>(),
                        allow_smem<__half, float>(), allow_smem<__half, __half>()})
    if (e != cudaSuccess) return e;
  return cudaSuccess;
}

SeqsGeom seqs_geom_simt(int64_t T, int group) {
  SeqsGeom g;
  g.group = group;
  g.tq = kR / group;
  g.bk = kK;
  g.slot_rows = (int)(g.tq < T ? g.tq : T) * group;
  g.ctas = 2 * current_device_sm_count();
  g.n_slots = 4 * g.ctas;
  g.min_tiles = 1;
  g.stream = 0;
  return g;
}

cudaError_t launch_seqs_simt(const SeqsArgs &a, const SeqsGeom &g, const SeqsSpace &s, cudaStream_t st) {
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
  const int64_t es = a.q.dtype == FM_F32 ? 4 : 2;
  const bool vec = quads(a.q, es) && quads(a.k, es) && quads(a.v, es);
  if (a.q.dtype == FM_F32) return launch_elem<float>(p, vec, st);
  if (a.q.dtype == FM_BF16) return launch_elem<__nv_bfloat16>(p, vec, st);
  return launch_elem<__half>(p, vec, st);
}

}  // namespace fm
