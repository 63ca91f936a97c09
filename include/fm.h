/*
 * fm.h -- C ABI of the fixed-m (const-max) attention forward for GB300 (sm_103a).
 *
 * The method replaces softmax's running row maximum by a shift fixed before any
 * score is computed, so that the base-2 numerator and denominator of every row
 * build up as plain fp32 sums across KV chunks, with one divide at the end.
 * Page references (title, section):
 *   [NKI]   "Kernel reference: ring_attention_const_max_fwd const-max ring attention"
 *   [PR477] "feat(attention): fixed-m splash attention kernel with dynamic bounds and
 *            safety fallbacks" (maxdiffusion PR #477)
 *   [PR478] "feat(attention): 2D Ulysses+Ring attention with Global Virtual
 *            K-Centering" (maxdiffusion PR #478)
 *
 * Call sequence for one attention forward over a key sequence split into chunks
 * (the ring's KV steps, run one after another on one GPU):
 *     fm_bounds(q, k_full, v_full)                       once
 *     fm_attn_chunk(q, k_c, v_c, accumulate = c > 0)     once per chunk c
 *     fm_finalize(acc_o, acc_sum -> o)                   once
 * or, fusing the last two: fm_attn_chunk_final(..., o) for the last chunk.
 * With key sinks (opts.sink_keys > 0) the loudest keys of each head are left out of the
 * key max and out of the chunks' fixed-m sums, and fm_fold_sinks merges them back exactly
 * after the last chunk (fm_attn_chunk_final and fm_attn_chunks with o_out do this
 * themselves).
 *
 * Conventions shared by every call:
 *   - Tensors are described by fm_tensor: a logical [B, H, S, D] array with element
 *     strides (any order, e.g. [B,H,S,D] or the pages' token-major [B,S,H,D]).
 *   - All buffers are device memory owned by the caller; the library allocates
 *     nothing and keeps no state besides a thread-local error string and one
 *     device-side error word per GPU.
 *   - Calls validate on the host, enqueue kernels on `stream` and return without
 *     synchronising.  On any error code nothing is enqueued and no output buffer is
 *     touched; fm_last_error() returns a message for the calling thread.
 *   - Device-side failures (a pipeline wait that exceeded its time limit) are
 *     reported by fm_sync_status().
 */
#ifndef FM_H_
#define FM_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define FM_API __attribute__((visibility("default")))
#else
#define FM_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st *fm_stream_t;

/* Element types.  The fixed-m calls accept only FM_F32 and FM_BF16: [PR477]'s commit message
 * rejects fp16 (and fp8) because 2^C-scale terms overflow their exponent range
 * (Q = K = 0, V = 1 gives inf instead of 1.0); here they fail with FM_ERR_DTYPE.  The calls over
 * requests of different lengths (end of this file) keep a running row max and take FM_F16 too. */
enum { FM_F32 = 0, FM_BF16 = 1, FM_F16 = 2, FM_F8E4M3 = 3, FM_F8E5M2 = 4 };

/* Return codes. */
enum {
  FM_OK = 0,
  FM_ERR_ARG = 1,             /* NULL pointer, negative size, bad flag value */
  FM_ERR_SHAPE = 2,           /* shapes of q / k / v / outputs disagree */
  FM_ERR_DTYPE = 3,           /* fp16 / fp8, or q, k, v of different types */
  FM_ERR_UNSUPPORTED = 4,     /* D not in {64, 128}; GQA (k.H != q.H); misaligned data */
  FM_ERR_BOUNDS_MISMATCH = 5, /* bounds do not belong to this call (see fm_attn_chunk) */
  FM_ERR_CUDA = 6,            /* a CUDA runtime call or kernel launch failed */
  FM_ERR_TIMEOUT = 7,         /* a kernel's pipeline wait ran past its limit */
  FM_ERR_INDEX = 8            /* fm_sync_status: an index in device memory was out of range (a page
                                 table entry, a cache slot, request lengths), and in debug builds
                                 (FM_DEBUG) a kernel's index check failed */
};

#define FM_BOUNDS_MAGIC 0x314D4246u /* tag written by fm_bounds ("FBM1") */
#define FM_BOUNDS_LOCAL_MAGIC 0x314C4246u /* fm_bounds_local done, fm_bounds_combine pending ("FBL1") */
#define FM_BLOCK_Q 128              /* rows per Q-block: the granularity of m and flag */
#define FM_VMAX 256                 /* the V bound of [PR477]'s commit message */
#define FM_SUM_CLAMP 1e-37f         /* [NKI] "Accumulate, then normalize once" */
#define FM_MAX_SINKS 8              /* most key sinks per head (opts.sink_keys) */

/* A logical [B, H, S, D] tensor: element (b,h,s,d) lives at
 * ptr + (b*stride[0] + h*stride[1] + s*stride[2] + d*stride[3]) * elemsize. */
typedef struct {
  void *ptr;
  int32_t dtype; /* FM_F32 or FM_BF16 */
  int32_t reserved;
  int64_t B, H, S, D;
  int64_t stride[4]; /* element strides, >= 0 */
} fm_tensor;

typedef struct {
  float softmax_scale;  /* <= 0 selects 1/sqrt(D) ([NKI] Interface table) */
  int32_t centering;    /* 1: virtual K-centering ([PR477] "Virtual K-centering") */
  int32_t force_online; /* 1: every Q-block takes the online-softmax fallback */
  int32_t per_row;      /* 1: each query row gets its own shift m_i = ceil(U_i) - C, with
                           U_i = alpha*|q_i|*max|k| ([NKI] "Best practices": give each query
                           row its own bound); 0: one m per 128-row Q-block ([PR477]).
                           Eligibility stays per Q-block in both cases. */
  int32_t sink_keys;    /* 0..FM_MAX_SINKS: leave up to this many of each head's loudest
                           keys out of the key max ([NKI] "Adapting this kernel": attention
                           sinks inflate max|k| for every row, and excluding those few keys
                           from the max reduction recovers the bound).  The sinks are the
                           keys whose norm (|k - kbar| with centering) is strictly above the
                           (sink_keys+1)-th largest, so ties at that norm stay ordinary keys;
                           kmax_sq becomes that norm squared.  The chunks skip the sinks and
                           fm_fold_sinks merges them back exactly, so the output is still
                           plain attention over every key. */
  int32_t schedule;     /* how the tensor-core chunk kernel spreads its work (FM_SCHEDULE_*);
                           the result is the same bits either way.  Ignored by fm_bounds. */
} fm_opts;

/* fm_opts.schedule.  A work item is two 128-row Q tiles of one (batch, head) against every key
 * tile of the call.  GRID launches one CTA per item.  PERSISTENT launches one CTA per SM that
 * walks the items in turn, loading the next item's Q and K/V tiles and running its first S
 * MMAs while the softmax warps finish the current item's epilogue (its K/V ring has one stage
 * fewer; that space stages O for the bulk accumulator add; the CTAs with one item fewer start
 * spread over an item's time, so that the CTAs' epilogues do not all meet the memory system at
 * once).  AUTO takes PERSISTENT when the
 * call has at most 8 key tiles (1024 keys) and at least twice as many items as the GPU has SMs,
 * GRID otherwise: measured on GB300, the overlap pays on such short items and the simpler grid
 * wins on longer ones. */
enum { FM_SCHEDULE_AUTO = 0, FM_SCHEDULE_GRID = 1, FM_SCHEDULE_PERSISTENT = 2 };

/* Bounds of one attention call ([PR477] Summary, "Dynamic eligibility bounding").
 * The caller allocates the device arrays and fills the pointers; fm_bounds fills
 * every other field.  nqb = ceil(Sq / FM_BLOCK_Q).
 *   m       int32 [B, H, nqb]  per-(head, Q-block) shift m = ceil(U) - C(N)
 *   flag    uint8 [B, H, nqb]  1 = eligible for fixed-m: v_ok && U <= gate
 *   qmax_sq f32   [B, H, nqb]  max over the block's rows of ||q_i||^2
 *   kmax_sq f32   [B, H]       max_j ||k_j - kbar||^2 (centered) or ||k_j||^2, over the
 *                              keys that are not sinks
 *   kbar    f32   [B, H, D]    mean key over all real keys ([PR478] Summary); 0 if
 *                              not centering
 *   qkbar   f32   [B, H, Sq]   alpha * q_i . kbar, the per-row centering term; 0 if not
 *                              centering
 *   shift   f32   [B, H, Sq]   the row's whole base-2 shift b_i = m_i + qkbar_i, with m_i
 *                              the row's own ceil(U_i) - C (opts.per_row) or its Q-block's
 *                              m; the chunk kernels subtract it in registers
 *   vmax_sq f32   [1]          max over all of V of v^2 (v_ok = vmax_sq <= 256^2)
 *   sink_idx int32 [B, H, FM_MAX_SINKS]  global key indices of the head's sinks, ascending,
 *                              padded with INT32_MAX (only with opts.sink_keys > 0)
 *   sink_k, sink_v f32 [B, H, FM_MAX_SINKS, D]  the sinks' raw key and value rows (zero in
 *                              padding slots), kept for fm_fold_sinks (sink_keys > 0 only)
 * with alpha = softmax_scale * log2(e) (base-2 logits, [PR477]'s exp2 formulation)
 * and U = alpha * sqrt(qmax_sq) * sqrt(kmax_sq), the Cauchy-Schwarz bound on the
 * base-2 logit ([NKI] "Picking a max that is safe without measuring it"). */
typedef struct {
  int32_t *m;
  uint8_t *flag;
  float *qmax_sq;
  float *kmax_sq;
  float *kbar;
  float *qkbar;
  float *shift;
  float *vmax_sq;
  int32_t *sink_idx; /* required when opts.sink_keys > 0, else ignored (may be NULL) */
  float *sink_k;
  float *sink_v;
  /* filled by fm_bounds */
  int64_t B, H, Sq, D, n_qblocks;
  int64_t N_total;   /* total KV length over every chunk of the call */
  int32_t C, W, gate; /* C(N) = 127 - ceil(log2 N) - 8, W = C + 125, gate = floor(W/2) */
  int32_t centered;  /* the opts.centering the bounds were measured with */
  int32_t per_row;   /* the opts.per_row they were built with */
  int32_t n_sink;    /* the opts.sink_keys they were built with */
  float alpha;
  int32_t dtype;
  /* updated by fm_attn_chunk (host-side bookkeeping of the chunk sequence) */
  int64_t kv_seen;
  int64_t next_key_offset; /* -1 (as fm_bounds / fm_bounds_combine and every chunk call leave it):
                              the next chunk's first key has global index kv_seen (0 with
                              accumulate = 0), i.e. the chunks come in key order.  A caller that
                              folds them in another order -- a ring hands rank r the shards in
                              the rotated order r, r-1, ... -- sets it to the chunk's global offset
                              before the call.  Only key sinks depend on it (they are found by
                              global key index). */
  int32_t online_lock;
  int32_t sinks_folded; /* set by fm_fold_sinks; no chunk may follow it */
  uint32_t magic; /* FM_BOUNDS_MAGIC once fm_bounds has succeeded */
} fm_bounds_out;

/* Scratch bytes fm_bounds needs for k_full of shape [B, H, N_total, D] (partial
 * key sums for the mean, per-block key and value maxima, per-block key-sink candidates).
 * Returns FM_OK. */
FM_API int fm_bounds_workspace_size(int64_t B, int64_t H, int64_t N_total, int64_t D, size_t *bytes);

/* fm_bounds -- norms, key mean, m and the per-tile flag ([PR477] Summary; the
 * fused norm reduction of [NKI] "Transpose prologue with fused norms" and [PR478]).
 *   q      [B, H, Sq, D]  queries (all rows of the call)
 *   k_full [B, H, N, D]   ALL keys of the call (every chunk), N = N_total
 *   v_full [B, H, N, D]   all values
 *   opts   softmax_scale, centering, per_row, sink_keys (force_online is ignored here)
 *   out    caller-filled pointers; every other field is written
 *   workspace, workspace_bytes  device scratch of at least fm_bounds_workspace_size
 * Device results are deterministic (fixed-order reductions; key-sink ties broken by the
 * lower index).  Errors: FM_ERR_ARG (also sink_keys outside [0, FM_MAX_SINKS] or a missing
 * sink array), FM_ERR_SHAPE, FM_ERR_DTYPE, FM_ERR_UNSUPPORTED (also sinks with N_total
 * above 2^31 - 256), FM_ERR_CUDA. */
FM_API int fm_bounds(const fm_tensor *q, const fm_tensor *k_full, const fm_tensor *v_full,
              const fm_opts *opts, fm_bounds_out *out, void *workspace, size_t workspace_bytes,
              fm_stream_t stream);

/* fm_attn_chunk -- fold one KV chunk into the unnormalised fp32 accumulators
 * ([NKI] "A static bound makes the ring reduction pure addition", "Accumulate, then
 * normalize once").  For an eligible Q-block (flag = 1, force_online = 0) each row i
 * adds p_ij = 2^(alpha*q_i.k_j - shift_i) to acc_sum and p_ij*v_j to acc_o: pure
 * addition across chunks.  Other Q-blocks take the online-softmax fallback ([PR478]
 * "Cross-Ring Safety Fallback"): a running row max kept in acc_max, with rescaling.
 *   q        [B, H, Sq, D]   the same queries given to fm_bounds
 *   k_chunk  [B, H, Nc, D]   this chunk's keys (Nc >= 0, any Nc, ragged tails allowed)
 *   v_chunk  [B, H, Nc, D]
 *   bounds   from fm_bounds for this call; kv_seen/online_lock are updated
 *   acc_o    f32 [B, H, Sq, D] contiguous;  acc_sum, acc_max f32 [B, H, Sq] contiguous.
 *            acc_max holds each row's current base-2 shift (shift_i on fixed-m rows,
 *            the running max on fallback rows), so acc_sum * 2^acc_max is the
 *            row's sum of 2^z.
 *   accumulate  0: overwrite the accumulators (first chunk); 1: add into them
 * Key sinks (bounds->n_sink > 0): a key whose global index is in bounds->sink_idx adds
 * nothing here.  The global index of a chunk's first key is bounds->next_key_offset when the
 * caller set it (chunks in any order, e.g. a ring's rotated order), else the number of keys
 * folded before it (bounds->kv_seen: chunks in the key order fm_bounds saw).
 * Errors: FM_ERR_BOUNDS_MISMATCH when bounds->magic is wrong, the bounds' shape is
 * not [B, H, ceil(Sq/128)], bounds->centered != opts->centering (raw-key bounds must
 * never pair with centered logits: [PR477] "matched pair"), the softmax scale
 * differs, more keys arrive than bounds->N_total (or, at the chunk's offset, lie past it),
 * force_online changes within a call,
 * opts->sink_keys differs from bounds->n_sink, or the sinks were already folded in
 * (accumulate = 1 after fm_fold_sinks); plus the errors of fm_bounds. */
FM_API int fm_attn_chunk(const fm_tensor *q, const fm_tensor *k_chunk, const fm_tensor *v_chunk,
                  fm_bounds_out *bounds, const fm_opts *opts, float *acc_o, float *acc_sum,
                  float *acc_max, int accumulate, fm_stream_t stream);

/* fm_attn_chunk_final -- fold the LAST KV chunk and normalise in the same pass ([NKI]
 * "The ring loop": the last step folds and normalises, so the output write hides behind
 * attention instead of running as a separate tail).  Same arguments and checks as
 * fm_attn_chunk, plus
 *   o_out  [B, H, Sq, D] FM_F32 or FM_BF16 (any strides): o = acc / max(acc_sum, 1e-37)
 *   lse    f32 [B, H, Sq] contiguous, or NULL: as written by fm_finalize_lse
 * acc_sum and acc_max are updated as by fm_attn_chunk; acc_o is NOT (its contents are
 * unspecified afterwards).  The result equals fm_attn_chunk followed by fm_finalize (or
 * fm_finalize_lse); the tensor-core kernel does both in one launch where the layout of
 * o_out allows 16-byte stores, otherwise the two steps run back to back.  With key sinks
 * the chunk is folded as by fm_attn_chunk, then one pass merges the sinks back and
 * normalises (the result of fm_fold_sinks followed by fm_finalize(_lse)). */
FM_API int fm_attn_chunk_final(const fm_tensor *q, const fm_tensor *k_chunk, const fm_tensor *v_chunk,
                               fm_bounds_out *bounds, const fm_opts *opts, float *acc_o, float *acc_sum,
                               float *acc_max, int accumulate, const fm_tensor *o_out, float *lse,
                               fm_stream_t stream);

/* fm_attn_chunks -- fold n_chunks consecutive KV chunks (1..FM_MAX_CHUNKS) in one pass, and
 * with o_out given normalise after the last one.  The result equals fm_attn_chunk on each
 * chunk in order (the first with `accumulate`, the rest adding), followed by fm_finalize /
 * fm_finalize_lse when o_out is given; acc_o is then left unspecified, as with
 * fm_attn_chunk_final.  On the tensor-core path one launch walks every chunk's key tiles
 * (each with its own ragged end) and O and the row sums stay on chip across the chunk
 * boundaries, as the accumulator stays resident for the whole ring in [NKI] ("A static
 * bound makes the ring reduction pure addition").  k_chunks / v_chunks: arrays of n_chunks
 * fm_tensor [B, H, Nc, D].  Errors: those of fm_attn_chunk_final, FM_ERR_ARG for n_chunks
 * outside [1, FM_MAX_CHUNKS]. */
#define FM_MAX_CHUNKS 8
FM_API int fm_attn_chunks(const fm_tensor *q, const fm_tensor *k_chunks, const fm_tensor *v_chunks,
                          int n_chunks, fm_bounds_out *bounds, const fm_opts *opts, float *acc_o,
                          float *acc_sum, float *acc_max, int accumulate, const fm_tensor *o_out,
                          float *lse, fm_stream_t stream);

/* fm_finalize -- o = acc_o / max(acc_sum, 1e-37) ([NKI] "Accumulate, then normalize
 * once": one divide, sum floored near the smallest fp32 normal).
 *   acc_o f32 [B, H, Sq, D] and acc_sum f32 [B, H, Sq], contiguous
 *   o_out [B, H, Sq, D] (its B, H, S, D give the shape), FM_F32 or FM_BF16, any strides
 * Errors: FM_ERR_ARG, FM_ERR_DTYPE, FM_ERR_CUDA. */
FM_API int fm_finalize(const float *acc_o, const float *acc_sum, const fm_tensor *o_out,
                fm_stream_t stream);

/* fm_finalize_lse -- fm_finalize that also writes each row's log-sum-exp of the scaled
 * scores, lse_i = ln(sum_j exp(softmax_scale * q_i.k_j)), for training and for merging
 * partial results ([NKI] Interface: with training the kernel also returns
 * lse = c_i + log(sum_exp)).  Since acc_max holds each row's base-2 shift on both paths,
 * lse_i = ln(2) * (acc_max_i + log2(acc_sum_i)); a row that saw no key gets -inf.
 *   acc_max f32 [B, H, Sq] contiguous (as left by fm_attn_chunk)
 *   lse     f32 [B, H, Sq] contiguous, written
 * Errors: those of fm_finalize. */
FM_API int fm_finalize_lse(const float *acc_o, const float *acc_sum, const float *acc_max,
                           const fm_tensor *o_out, float *lse, fm_stream_t stream);

/* fm_fold_sinks -- merge the key sinks that fm_bounds set aside back into the accumulators,
 * exactly, after the last chunk and before fm_finalize(_lse) ([NKI] "Adapting this kernel"
 * leaves the loudest keys out of the max reduction; this is how their terms still count).
 * For each row i, with z_s = alpha * q_i.k_s the raw base-2 logit of sink s (from
 * bounds->sink_k) and r_i = acc_max_i the row's current shift:
 *   r' = max(r_i, max_s z_s),  c = 2^(r_i - r'),
 *   acc_o_i = c * acc_o_i + sum_s 2^(z_s - r') v_s,  acc_sum_i = c * acc_sum_i + sum_s 2^(z_s - r'),
 *   acc_max_i = r'
 * (an online-softmax merge in fp32), so that acc_sum * 2^acc_max stays the row's sum of 2^z
 * and fm_finalize_lse stays valid.  A no-op when bounds->n_sink == 0.
 *   q, opts  as given to the chunks;  acc_o / acc_sum / acc_max  as left by the last chunk
 * Errors: FM_ERR_BOUNDS_MISMATCH (bounds not matching q or opts, no chunk folded yet, or the
 * sinks already folded), FM_ERR_ARG, FM_ERR_CUDA. */
FM_API int fm_fold_sinks(const fm_tensor *q, fm_bounds_out *bounds, const fm_opts *opts, float *acc_o,
                         float *acc_sum, float *acc_max, fm_stream_t stream);

/* fm_sync_status -- synchronise `stream`, then report and clear this GPU's device
 * error word: FM_ERR_TIMEOUT if a kernel gave up on a pipeline wait (its outputs are
 * then invalid), FM_ERR_INDEX if a paged call met a page table entry, slot or length outside its
 * tensors or a debug build's index check failed (the library built with
 * -DFM_DEBUG: the chunk kernels check their epilogue accesses to the accumulators and o, skip
 * a failing one and record the first), FM_ERR_CUDA on an asynchronous CUDA error, else FM_OK. */
FM_API int fm_sync_status(fm_stream_t stream);

/* fm_probe_wait_timeout -- exercise the failure path of the kernels' bounded waits: one
 * thread waits on a barrier phase that nothing completes and gives up after timeout_ms
 * (1..10000), recording the failure in the device error word, so that the next
 * fm_sync_status returns FM_ERR_TIMEOUT (role 5) and clears it.  Nothing faults and the
 * context stays usable.  No counterpart in the pages: it tests the library's own failure
 * detection.  Errors: FM_ERR_ARG, FM_ERR_CUDA. */
FM_API int fm_probe_wait_timeout(unsigned int timeout_ms, fm_stream_t stream);

/* Message of the last failing call on this thread ("" if none).  Valid until the
 * thread's next fm_* call. */
FM_API const char *fm_last_error(void);

/* ABI version of this header: (major << 16) | minor.  1.2 added fm_opts.schedule,
 * fm_bounds_out.next_key_offset and the ring bounds calls; 1.3 the calls over requests of
 * different lengths and the paged cache. */
FM_API int fm_version(void);

/* ---- The bounds of a ring of ranks ---------------------------------------------------------
 * In a multi-GPU ring each rank keeps its own query rows and holds one shard of the keys and
 * values; the shards rotate through the ranks, so no rank ever sees all keys at once.  The bounds
 * still need ring-wide key statistics, and the pages exchange them once before the ring: the key
 * mean over real tokens reduced across the ring so every rank centers against the same mean
 * ([PR478] Summary, "Global Virtual K-Centering"), then one max-reduction of the per-head key
 * norms and the V maximum ([NKI] "Global key max"; [PR478] folds the centered key max and the V
 * max into one pmax).  The library computes each rank's part and combines the exchanged parts;
 * the caller moves the bytes with its own collectives:
 *   1. (centering only) fm_ring_key_sums(k_shard) -> ksum f32 [B, H, D], the shard's key sums;
 *      the caller all-reduces (sum) ksum over the ring;
 *   2. fm_bounds_local(q, k_shard, v_shard, key_offset, N_total, ksum) -> the query-side arrays
 *      of `out` and this rank's statistics block (fm_ring_stats_bytes bytes); the caller
 *      all-gathers the blocks, in rank order, into one buffer;
 *   3. fm_bounds_combine(stats_all, n_ranks) -> the rest of `out`: kmax_sq, vmax_sq, the key
 *      sinks, m, flag and shift, as fm_bounds would give over (q, every key, every value), up to
 *      the fp32 summation order of the key mean (m and flag can then differ only where U is
 *      within fp32 rounding of an integer or of the gate).
 * Every rank then folds the shards with fm_attn_chunk in ring order, setting
 * out->next_key_offset to each shard's global offset.  The statistics block holds, per head, the
 * shard's key max and, with key sinks, its sink_keys + 1 loudest keys (norm, global index, key
 * and value rows): the ring-wide loudest keys are among the union of those. */

/* Bytes of one rank's statistics block for q of [B, H, *, D] and opts.sink_keys.  Returns FM_OK. */
FM_API int fm_ring_stats_bytes(int64_t B, int64_t H, int64_t D, int sink_keys, size_t *bytes);

/* fm_ring_key_sums -- ksum[b,h,:] = sum of this rank's keys of (b, h) in fp32 (fixed order).
 *   k_shard [B, H, Nr, D];  ksum f32 [B, H, D] device, written;
 *   workspace of fm_bounds_workspace_size(B, H, Nr, D) bytes.
 * Errors: FM_ERR_ARG, FM_ERR_DTYPE, FM_ERR_UNSUPPORTED, FM_ERR_CUDA. */
FM_API int fm_ring_key_sums(const fm_tensor *k_shard, float *ksum, void *workspace, size_t workspace_bytes,
                            fm_stream_t stream);

/* fm_bounds_local -- this rank's part of the bounds.
 *   q        [B, H, Sq, D] this rank's queries
 *   k_shard, v_shard [B, H, Nr, D] its shard of the keys and values; key_offset = the global
 *            index of the shard's first key (0 <= key_offset, key_offset + Nr <= N_total)
 *   N_total  keys over every shard of the ring (C(N) is computed from it)
 *   ksum_total f32 [B, H, D]: the ring-wide key sums (step 1) when opts->centering, else NULL
 *   out      as for fm_bounds; the query-side arrays (qmax_sq, qkbar, kbar) are written here, the
 *            rest by fm_bounds_combine; out->magic becomes FM_BOUNDS_LOCAL_MAGIC
 *   stats    device buffer of fm_ring_stats_bytes bytes, written (16-byte aligned)
 *   workspace of fm_bounds_workspace_size(B, H, Nr, D) bytes
 * Errors: those of fm_bounds, FM_ERR_ARG for a bad key_offset / N_total or a missing ksum_total. */
FM_API int fm_bounds_local(const fm_tensor *q, const fm_tensor *k_shard, const fm_tensor *v_shard, int64_t key_offset,
                           int64_t N_total, const float *ksum_total, const fm_opts *opts, fm_bounds_out *out,
                           void *stats, void *workspace, size_t workspace_bytes, fm_stream_t stream);

/* fm_bounds_combine -- finish `out` from every rank's statistics block.
 *   stats_all  device buffer of n_ranks blocks of fm_ring_stats_bytes bytes, in rank order
 *   opts       the same opts as fm_bounds_local
 *   out        as left by fm_bounds_local on this rank; becomes ready for fm_attn_chunk
 * Errors: FM_ERR_BOUNDS_MISMATCH when out was not prepared by fm_bounds_local or opts differ,
 * FM_ERR_ARG, FM_ERR_CUDA. */
FM_API int fm_bounds_combine(const void *stats_all, int n_ranks, const fm_opts *opts, fm_bounds_out *out,
                             fm_stream_t stream);

/* ---- Whole forwards on host buffers --------------------------------------------------------
 * Device buffers of fm_attention_host, all owned by the caller: two sets of inputs and outputs,
 * which consecutive batches alternate between, and one set of accumulators, bounds and workspace,
 * which the batches reuse in order. */
typedef struct {
  fm_tensor q[2], k[2], v[2]; /* device, contiguous [B, H, Sq, D] / [B, H, N, D], the inputs' dtype */
  fm_tensor o[2];             /* device, contiguous [B, H, Sq, D], the outputs' dtype */
  float *acc_o, *acc_sum, *acc_max;
  fm_bounds_out *bounds;      /* host struct whose device arrays are set, as for fm_bounds */
  void *workspace;
  size_t workspace_bytes;
} fm_host_buffers;

/* fm_attention_host -- n_batches whole forwards whose inputs and outputs live in host memory.
 * For batch i: q_host[i], k_host[i], v_host[i] are copied to the device, the path runs
 * (fm_bounds, one fm_attn_chunk per chunk of chunk_lens, the last chunk fused with the
 * normalise), and o is copied back into o_host[i].  Batch i+1's upload and batch i-1's read-back
 * run on their own streams while batch i computes, so the copies hide behind the kernels (host
 * memory must be page-locked for that; pageable memory works but does not overlap).
 *   q_host, k_host, v_host, o_host  arrays of n_batches contiguous host tensors, shaped and typed
 *                  like the device buffers
 *   chunk_lens     n_chunks >= 1 key counts summing to N (the ring steps run one after another)
 *   streams        three caller-created streams: upload, compute, read-back
 * Returns when every output is in host memory.  Creates and destroys a few CUDA events; allocates
 * no device memory.  Errors: those of the calls it makes, FM_ERR_ARG / FM_ERR_SHAPE for buffers
 * that do not match, FM_ERR_UNSUPPORTED for non-contiguous ones. */
FM_API int fm_attention_host(const fm_tensor *q_host, const fm_tensor *k_host, const fm_tensor *v_host,
                             const fm_tensor *o_host, int n_batches, const int64_t *chunk_lens, int n_chunks,
                             const fm_opts *opts, const fm_host_buffers *dev, const fm_stream_t *streams);

/* Upper bound of the scratch fm_bounds_noalloc can use: 4 MiB.  That covers, at D = 128,
 * up to 74 heads of 75,600 keys (fm_bounds_workspace_size gives the exact need). */
#define FM_NOALLOC_SCRATCH_BYTES ((size_t)4 << 20)

/* fm_bounds_noalloc -- fm_bounds for callers that cannot allocate device memory.
 * The pages have no counterpart to this call: it exists for callers whose device memory
 * is planned in full before they run (an inference engine that reserves its arena up
 * front and forbids allocation afterwards, a plug-in inside another framework's memory
 * pool) and for latency-critical streams that must not pay cudaMalloc's implicit device
 * synchronisation.  Same arguments and results as fm_bounds, minus the workspace: the
 * scratch lives in a file-scope device array of FM_NOALLOC_SCRATCH_BYTES inside libfm,
 * which every GPU that loads the library holds until the process exits.
 *   - Nothing is allocated: no cudaMalloc, cudaFree or allocating library routine.
 *   - The first call on each device looks up the array's device address with that device
 *     current (cudaGetSymbolAddress); make that first call before any stream capture.
 *   - Every call shares the one array and it keeps the last call's contents; nothing in
 *     it needs to start at zero, since every slot the kernels read is written earlier in
 *     the same call.  Calls that overlap on the GPU (other streams, other threads) race
 *     on it: serialise them.
 * Errors: those of fm_bounds, plus FM_ERR_UNSUPPORTED when the problem needs more scratch
 * than FM_NOALLOC_SCRATCH_BYTES (nothing is enqueued then). */
FM_API int fm_bounds_noalloc(const fm_tensor *q, const fm_tensor *k_full, const fm_tensor *v_full,
                             const fm_opts *opts, fm_bounds_out *out, fm_stream_t stream);

/* ---- Requests of different lengths, and a paged key/value cache ------------------------------
 * Attention for serving causal models: n requests, each with its own number of queries and keys,
 * in one call.  Not fixed-m (the pages' bound is per dense call): every row keeps a running max.
 *   - Packed tensors hold every request's rows one after another: [1, H, T, D], request i owning
 *     rows cu[i] .. cu[i+1]-1 (cu int32 [n+1], cu[0] = 0, ascending).  Rows behind the last
 *     request are neither read nor written.
 *   - A paged cache is [num_pages, H, page_size, D]; position p of request i lies in page
 *     block_table[i][p / page_size], row p % page_size.  Table entries past a request's last key
 *     are not read.  Any strides; a page is shared by requests when their tables say so.
 *   - Query heads share key heads: head h reads key head h / (Hq / Hk); Hq a multiple of Hk, at
 *     most FM_MAX_GROUP to one.
 *   - With q_i queries and s_i keys, query t of request i stands at position p = s_i - q_i + t.
 *     causal: it sees keys j <= p; window > 0 (needs causal): only j > p - window.  A row that sees
 *     no key gets o = 0 and lse = -inf.
 *   - FM_F32, FM_BF16 or FM_F16, one type for q, k, v; sums, the row max and the normalise are fp32.
 *   - 16-bit types run on the tensor cores, where the weights p are rounded to that type before they meet v,
 *     if every tensor's innermost stride is 1, its address and other strides are multiples of 16 bytes, no
 *     stride of more than one element is 0 (a head expanded to several) and a page has 8, 16, 32, 64 or a
 *     multiple of 128 rows.  Other 16-bit layouts and fp32 run on the CUDA cores, several times slower; p is
 *     fp32 there.
 *   - How the work is cut is chosen from the arrays' sizes (T, n_seqs, heads), since the lengths are
 *     on the device.  Rows of q that no request owns and requests without queries change no result but
 *     cost time: little on the tensor cores, up to five times for fp32 decoding in buffers far longer than its
 *     rows.
 *   - Keys and values that no query of the request sees (past its end in its last page, its
 *     neighbours' rows, before every query's window) may hold anything, NaN too: they change
 *     nothing, and table entries of pages before the window are not read.  A value row that some
 *     query of the request sees must be finite: a NaN or infinity there may reach that request's
 *     other rows.
 *   - All lengths are read on the device: nothing waits for them, calls can be captured into a
 *     graph and replayed with other lengths (the first call on a device comes before any
 *     capture).  Lengths that do not fit the tensors are clamped, cu_q that runs backwards computes
 *     nothing, a table entry outside [0, num_pages) reads as zeros, and the next fm_sync_status
 *     returns FM_ERR_INDEX; it does so too after a decoding call of more than about 4e8 tiles
 *     (128 keys of one key head each; some 5 s of work), which computes nothing.
 *   - The workspace is scratch: its contents need no preparation and mean nothing afterwards.  Calls
 *     that may run at the same time need one each. */
#define FM_MAX_GROUP 64
#define FM_MAX_SEQS 8192

typedef struct {
  float softmax_scale; /* <= 0 selects 1/sqrt(D) */
  int32_t causal;      /* 1 or 0 */
  int32_t window;      /* 0: none */
} fm_seqs_opts;

/* Device arrays of one attention call (host struct). */
typedef struct {
  int64_t n_seqs;             /* 0 .. FM_MAX_SEQS */
  const int32_t *cu_q;        /* [n+1] */
  const int32_t *cu_k;        /* [n+1], fm_attn_varlen */
  const int32_t *kv_len;      /* [n] keys of each request with its new tokens, fm_attn_paged */
  const int32_t *block_table; /* [n] rows of table_width entries, table_stride apart, fm_attn_paged */
  int64_t table_stride, table_width;
} fm_seqs;

/* Scratch bytes of fm_attn_varlen / fm_attn_paged for n requests, T packed query rows and the given
 * heads.  Never less for more requests or rows. */
FM_API int fm_attn_seqs_workspace_size(int64_t n_seqs, int64_t T, int64_t Hq, int64_t Hk, int64_t D, size_t *bytes);

/* fm_attn_varlen -- attention over packed keys: whole prompts of different lengths.
 *   q [1, Hq, T, D];  k, v [1, Hk, Tk, D];  seqs: n_seqs, cu_q, cu_k
 *   o_out [1, Hq, T, D], q's type or FM_F32;  lse f32 [Hq, T] contiguous or NULL (natural log)
 *   workspace of fm_attn_seqs_workspace_size bytes, 16-byte aligned (a part of a larger buffer will do)
 * Deterministic: the same call gives the same bits.  Errors: FM_ERR_ARG, FM_ERR_SHAPE, FM_ERR_DTYPE,
 * FM_ERR_UNSUPPORTED (D not 64 or 128, too many heads to a key head, requests or rows), FM_ERR_CUDA. */
FM_API int fm_attn_varlen(const fm_tensor *q, const fm_tensor *k, const fm_tensor *v, const fm_seqs *seqs,
                          const fm_seqs_opts *opts, const fm_tensor *o_out, float *lse, void *workspace,
                          size_t workspace_bytes, fm_stream_t stream);

/* fm_attn_paged -- the same over a paged cache that already holds the new tokens' keys and values:
 * one query a request (decoding), chunks of a prompt, or both in one call.
 *   k_cache, v_cache [num_pages, Hk, page_size, D];  seqs: n_seqs, cu_q, kv_len, block_table */
FM_API int fm_attn_paged(const fm_tensor *q, const fm_tensor *k_cache, const fm_tensor *v_cache, const fm_seqs *seqs,
                         const fm_seqs_opts *opts, const fm_tensor *o_out, float *lse, void *workspace,
                         size_t workspace_bytes, fm_stream_t stream);

/* ---- Trees of drafted tokens ------------------------------------------------------------------
 * A request's new tokens may be guesses that a cheaper model has drafted: the nodes of a tree, packed
 * like any new tokens (cu_q, their keys and values in the cache at consecutive positions).  Node 0 is
 * the last token that is certain; a node's children are guesses at the token after it.
 *   parent int32 [T]  the node's parent, counted from its request's first node: an earlier one, or -1
 *   mask              rows of mask_words 32-bit words, mask_stride words apart, one a token: bit j (of
 *                     word j / 32) of row t says that t sees node j of its request.  Bits of later
 *                     nodes (j > t) and of nodes that the request does not have are not looked at.
 * A request of more new tokens than a mask row has bits (a prompt chunk in the same call) is causal; a chunk of
 * fewer is a tree like any other, and causal where each token's parent is the one before it. */
#define FM_MAX_NODES 1024 /* bits of a mask row, and nodes of a tree that fm_tree_verify takes */

/* fm_tree_mask -- the mask of trees: every node sees itself and its ancestors.
 *   seqs       n_seqs, cu_q and kv_len (keys with the nodes counted) are used
 *   T          rows of parent, mask and positions; rows behind the last request are left as they are
 *   mask       uint32 written, mask_words 1 to FM_MAX_NODES / 32; rows of causal requests are set to 0
 *   positions  int32 [T] written, or NULL: kv_len - (new tokens) + the node's depth (of a causal
 *              request its place), the position that a rotary embedding wants
 * A parent that is not an earlier node is taken for -1 and reported by fm_sync_status (FM_ERR_INDEX), as
 * cu_q that does not fit T rows is.  Errors: FM_ERR_ARG, FM_ERR_UNSUPPORTED, FM_ERR_CUDA. */
FM_API int fm_tree_mask(const fm_seqs *seqs, const int32_t *parent, int64_t T, uint32_t *mask, int64_t mask_words,
                        int64_t mask_stride, int32_t *positions, fm_stream_t stream);

/* fm_attn_tree -- fm_attn_paged where each new token sees every key before its request's new tokens, and
 * of these the ones up to itself that its mask row names: the nodes of one request, of different
 * branches, in one call.  causal = 1, window = 0 (FM_ERR_ARG, FM_ERR_UNSUPPORTED otherwise).  A token
 * whose row is 0 and that has no earlier key gets o = 0 and lse = -inf.  Values of nodes that no row of a
 * mask names still have to be finite.  Workspace and errors as there. */
FM_API int fm_attn_tree(const fm_tensor *q, const fm_tensor *k_cache, const fm_tensor *v_cache, const fm_seqs *seqs,
                        const uint32_t *mask, int64_t mask_words, int64_t mask_stride, const fm_seqs_opts *opts,
                        const fm_tensor *o_out, float *lse, void *workspace, size_t workspace_bytes, fm_stream_t stream);

/* fm_tree_verify -- the nodes of each tree that the target model keeps, and the token after them.
 * Row t of target is the target's distribution of the token after node t, row t of draft the one that t's
 * children were drawn from, independently, whatever their number.  The walk begins at node 0 and tries a
 * node's children in order; with p, q the rows after the node that it stands at, A = 0 and S = 1 when it
 * comes there, a child of token x and number u is kept if
 *     u q(x) S < max(p(x) - A q(x), 0);  else A += S, S = sum_y max(p(y) - A q(y), 0)  (0: A = 0, S = 1).
 * draft NULL: the children were chosen, not drawn; one is kept if u S < p(x), else S -= p(x) (not below 0)
 * and p(x) = 0 for what follows at that node.  At a node that keeps no child the next token is the least x with
 * sum_{y <= x} R(y) > u_last sum_y R(y), R what is left there of p: max(p - A q, 0), or p without the
 * refused tokens (p itself where that leaves nothing).  With uniform numbers the tokens kept and the next
 * one are distributed as the target's own.
 *   target, draft  [1, 1, T, V], FM_F32, FM_BF16 or FM_F16 alike, adjacent along V, rows any distance apart.
 *              They are taken to sum to 1 and are not scaled.  What is negative, infinite or NaN counts as 0
 *   cu_q       int32 [n+1]: request i has nodes cu_q[i] .. cu_q[i+1]-1, at most FM_MAX_NODES
 *   tokens, parent  int32 [T]; a node whose parent is not an earlier one is never tried
 *   u          float [T], u_last float [n]: random numbers of [0, 1); 1 and more count as 1, NaN as 0
 *   max_path   1 to FM_MAX_NODES: the walk ends after so many nodes
 *   path       int32 [n, max_path] written: the nodes kept, node 0 first, -1 behind them
 *   kept       int32 [n] written: their number; 0 for a request without nodes
 *   next_token int32 [n] written: -1 for a request without nodes, or whose last row of p is all 0
 * Tests and sums are made in pairs of fp32 numbers, a value and its error, and the result is the definition's
 * unless a random number lies as close to a border as they are off: what is left of a token by at most
 * 2^-46 (p + A q), a sum over V tokens besides by at most (N^2 + N) 2^-48 sum (p + 2 A q), N = V / 1024 + 20 the
 * numbers that one of its lanes adds (on rows of softmaxes by 2^-48 up to V = 2^21, 2^-44 at 2^24).  A token
 * outside the vocabulary is never kept, more than FM_MAX_NODES nodes are none; fm_sync_status reports both
 * (FM_ERR_INDEX).
 * Rows of draft that lie otherwise to a 16-byte boundary than target's are read an element at a time, which takes
 * longer.  Errors: FM_ERR_ARG, FM_ERR_SHAPE, FM_ERR_DTYPE, FM_ERR_UNSUPPORTED, FM_ERR_CUDA. */
FM_API int fm_tree_verify(const fm_tensor *target, const fm_tensor *draft, int64_t n_seqs, const int32_t *cu_q,
                          const int32_t *tokens, const int32_t *parent, const float *u, const float *u_last,
                          int64_t max_path, int32_t *path, int32_t *kept, int32_t *next_token, fm_stream_t stream);

/* fm_tree_verify_rows -- the same in a step whose requests are not all trees: prompt chunks of any length beside them are
 * passed over, and only nodes have rows of probabilities.
 *   target, draft  [1, 1, R, V]: row rows[i] + t is the one after node t of request i
 *   rows       int32 [n]; negative: request i is not verified, whatever its tokens are.  Its path is all -1, its
 *              next_token -1 and kept -1, with which fm_paged_keep leaves all of them in the cache
 *   T          length of tokens, parent and u, where request i's are cu_q[i] .. cu_q[i+1]-1
 * Rows that target does not have: the request has no nodes, and fm_sync_status reports it (FM_ERR_INDEX). */
FM_API int fm_tree_verify_rows(const fm_tensor *target, const fm_tensor *draft, int64_t n_seqs, const int32_t *cu_q,
                               const int32_t *rows, int64_t T, const int32_t *tokens, const int32_t *parent, const float *u,
                               const float *u_last, int64_t max_path, int32_t *path, int32_t *kept, int32_t *next_token,
                               fm_stream_t stream);

/* The state of a paged cache's bookkeeping (host struct of device arrays). */
typedef struct {
  int64_t n_seqs, page_size, num_pages;
  int32_t *block_table; /* [n] rows of table_width entries, table_stride apart */
  int64_t table_stride, table_width;
  int32_t *free_pages;       /* [num_pages]: the free pages are its first free_count entries */
  const int32_t *free_count; /* [1] */
  int32_t *free_count_out;   /* [1], may be free_count */
  const int32_t *kv_len;     /* [n] tokens that each request holds */
  int32_t *kv_len_out;       /* [n], may be kv_len */
} fm_page_state;

/* fm_paged_extend -- room for the next tokens of every request: one launch where max_tokens is at most
 * 4,096, two beyond (the room decides, not the tokens; all of slots and positions is written each time).
 *   new_len   int32 [n]  tokens to come (0: none)
 *   release   uint8 [n] or NULL: 1 = the request that held row i has ended: its pages go back to
 *             the list first, and new_len[i] tokens begin a new request in that row
 *   max_tokens  length of slots and positions
 *   cu_q      int32 [n+1] written: prefix sums of new_len
 *   slots     int64 [max_tokens] written: page * page_size + row of each new token, in request
 *             order, -1 behind the last
 *   positions int32 [max_tokens] written: its position in its request, -1 behind the last
 *   status    int32 [1] written: 0, or the number of pages that the list is short of, or -1 (a
 *             negative length, lengths that the table row, max_tokens or 31 bits do not hold, a
 *             free_count outside the list).  Unless 0 the call changes nothing: lengths, count,
 *             table and list stay, cu_q is all 0 and slots and positions all -1, so that the
 *             cache write and the attention that follow do nothing.
 * Pages given back are put on the list's end in request and table order; new pages are taken from
 * its end.  A page belongs to one row here: a page that several tables share would be given back by
 * each of their rows, so such tables are kept by the caller.  Errors: FM_ERR_ARG, FM_ERR_UNSUPPORTED, FM_ERR_CUDA. */
FM_API int fm_paged_extend(const fm_page_state *state, const int32_t *new_len, const uint8_t *release,
                           int64_t max_tokens, int32_t *cu_q, int64_t *slots, int32_t *positions, int32_t *status,
                           fm_stream_t stream);

/* fm_paged_write -- k and v rows [1, H, T, D] put at their slots of the caches [num_pages, H,
 * page_size, D] (one dtype, any strides).  slots int64 [T]: a negative one skips its row, one past the
 * cache is skipped and reported by fm_sync_status (FM_ERR_INDEX).  Slots are distinct (of rows with
 * one slot, either may remain in each piece).  Errors: FM_ERR_ARG, FM_ERR_SHAPE, FM_ERR_DTYPE,
 * FM_ERR_UNSUPPORTED, FM_ERR_CUDA. */
FM_API int fm_paged_write(const fm_tensor *k, const fm_tensor *v, const int64_t *slots, const fm_tensor *k_cache,
                          const fm_tensor *v_cache, fm_stream_t stream);

/* fm_paged_keep -- the bookkeeping after fm_tree_verify: of each request's new tokens (the nodes of a tree, whose
 * keys and values are in the cache) only the path that was kept stays, as if it alone had been appended.
 *   state     kv_len: keys with the new tokens counted; kv_len_out: kv_len - (new tokens) + kept.  Pages that hold
 *             none of them go to the end of the list of free pages, in request and table order (their
 *             entries stay in the table, behind the request's last key)
 *   cu_q      int32 [n+1]: request i has cu_q[i+1] - cu_q[i] new tokens
 *   path      int32 [n, max_path], kept int32 [n]: the first kept[i] entries of path[i], ascending, are the new
 *             tokens that stay; 0: none does; -1: all do (a prompt chunk in the same call, which
 *             fm_tree_verify_rows passed over)
 *   src, dst  int64 [n, max_path] written: the slots that fm_paged_move reads and writes, -1 where nothing moves
 *   status    int32 [1] written: 0, or the number of requests whose kept or path cannot be (they keep all they
 *             have), or -1: free_count and the pages given back do not fit the list, and the call changes nothing
 * Errors: FM_ERR_ARG, FM_ERR_UNSUPPORTED, FM_ERR_CUDA. */
FM_API int fm_paged_keep(const fm_page_state *state, const int32_t *cu_q, int64_t max_path, const int32_t *path,
                         const int32_t *kept, int64_t *src, int64_t *dst, int32_t *status, fm_stream_t stream);

/* fm_paged_move -- one layer's rows of the tokens kept moved to their places, after fm_paged_keep and before the
 * next fm_paged_extend (the pages given back still hold rows).  src, dst int64 [n, max_path] from fm_paged_keep:
 * moves of one row are made in order, none reading what an earlier one wrote; rows do not share slots.  Negative
 * slots are skipped, ones past the cache too, and reported by fm_sync_status (FM_ERR_INDEX).
 *   k_cache, v_cache  [num_pages, H, page_size, D], any strides
 * Errors: FM_ERR_ARG, FM_ERR_SHAPE, FM_ERR_DTYPE, FM_ERR_UNSUPPORTED, FM_ERR_CUDA. */
FM_API int fm_paged_move(int64_t n_seqs, int64_t max_path, const int64_t *src, const int64_t *dst, const fm_tensor *k_cache,
                         const fm_tensor *v_cache, fm_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* FM_H_ */
