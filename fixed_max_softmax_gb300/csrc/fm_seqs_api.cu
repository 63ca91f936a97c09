// fm_seqs_api.cu -- the C ABI of the serving calls: attention over requests of different lengths
// (packed or paged keys) and the paged cache's bookkeeping.  As fm_api.cu: everything is checked on
// the host, nothing is enqueued on an error, nothing is allocated, nothing waits.
#include <limits.h>
#include <math.h>

#include <atomic>

#include "fm_internal.h"

using namespace fm;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 30;  // packed rows of one call: rows are indexed in 32 bits

// Validate one fm_tensor of these calls (fp32, bf16 or fp16) and turn it into a View.
int seqs_view(const fm_tensor *t, const char *what, View *v) {
  if (!t) return fail(FM_ERR_ARG, "%s: NULL tensor", what);
  if (t->dtype == FM_F8E4M3 || t->dtype == FM_F8E5M2) return fail(FM_ERR_DTYPE, "%s: fp8 is not supported", what);
  if (t->dtype != FM_F32 && t->dtype != FM_BF16 && t->dtype != FM_F16)
    return fail(FM_ERR_ARG, "%s: unknown dtype %d", what, t->dtype);
  if (t->B < 0 || t->H < 0 || t->S < 0 || t->D < 0)
    return fail(FM_ERR_ARG, "%s: negative dimension [%lld,%lld,%lld,%lld]", what, (long long)t->B, (long long)t->H,
                (long long)t->S, (long long)t->D);
  for (int i = 0; i < 4; ++i)
    if (t->stride[i] < 0) return fail(FM_ERR_ARG, "%s: negative stride", what);
  if (t->D != 64 && t->D != 128)
    return fail(FM_ERR_UNSUPPORTED, "%s: head dimension %lld not supported (64 or 128)", what, (long long)t->D);
  if (t->H > 65535) return fail(FM_ERR_UNSUPPORTED, "%s: H above 65535", what);
  if (t->S > kMaxRows || t->B > kMaxRows)
    return fail(FM_ERR_UNSUPPORTED, "%s: more than 2^30 rows or pages", what);
  const size_t es = t->dtype == FM_F32 ? 4 : 2;
  if (t->B * t->H * t->S > 0 && !t->ptr) return fail(FM_ERR_ARG, "%s: NULL data pointer", what);
  if (reinterpret_cast<uintptr_t>(t->ptr) % es) return fail(FM_ERR_UNSUPPORTED, "%s: misaligned data", what);
  *v = View{t->ptr, t->dtype, t->B, t->H, t->S, t->D, t->stride[0], t->stride[1], t->stride[2], t->stride[3]};
  return FM_OK;
}

bool misaligned(const void *p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

int check_group(int64_t Hq, int64_t Hk) {
  if (Hk < 1 || Hq < 1 || Hq % Hk) return fail(FM_ERR_SHAPE, "%lld query heads are not a multiple of %lld key heads", (long long)Hq, (long long)Hk);
  if (Hq / Hk > FM_MAX_GROUP)
    return fail(FM_ERR_UNSUPPORTED, "%lld query heads to a key head: at most %d", (long long)(Hq / Hk), FM_MAX_GROUP);
  return FM_OK;
}

// Rows of a unit of the CUDA-core kernels: 8 or 16 where most requests' rows of a key head fit them.  Judged by
// the arrays, as the lengths are on the device: fp32 decoding of 64 requests (5 heads to a key head) takes 371 us
// in buffers of 64 rows, 736 in 128 (16 rows a unit), 1,860 in 2,048 (64); a prompt of 500 alone 129, among 255
// idle rows 153.
int simt_rows(int64_t T, int64_t n, int group) {
  for (int rows = 8; rows <= 16; rows *= 2)
    if (group <= rows && T * group <= rows * n) return rows;
  return 64;
}

// The workspace is given at any 16-byte boundary and used from the next of kSpaceAlign: partial results are
// stored 32 bytes at a time, rows of theirs in whole 128-byte lines.
constexpr size_t kSpaceAlign = 128;

size_t space_bytes(int64_t n, int64_t T, int64_t Hq, int64_t Hk, int64_t D) {
  const int group = (int)(Hq / Hk);
  size_t most = seqs_space(seqs_geom_simt(T, group, 64), n, T, Hk, D).total;
  const size_t tc = seqs_space(seqs_geom_tc(T, n, group), n, T, Hk, D).total;
  if (tc > most) most = tc;
  for (int rows = 8; rows <= 16; rows *= 2) {
    if (group > rows) continue;
    // of as many tokens as a call with so few rows a request may have, so that no smaller call needs more
    const int64_t t = T * group <= rows * n ? T : rows * n / group;
    const size_t few = seqs_space(seqs_geom_simt(t, group, rows), n, t, Hk, D).total;
    if (few > most) most = few;
  }
  return most + kSpaceAlign - 16;
}

// Every attention kernel's attributes, at the first call on the current device.
cudaError_t prepare() {
  constexpr int kDevices = 64;
  static std::atomic<bool> ready[kDevices] = {};  // set by whichever thread is first, or by several
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev >= 0 && dev < kDevices && ready[dev])) return e;
  if ((e = seqs_plan_prepare()) != cudaSuccess || (e = seqs_simt_prepare()) != cudaSuccess ||
      (e = seqs_tc_prepare()) != cudaSuccess)
    return e;
  if (dev >= 0 && dev < kDevices) ready[dev] = true;
  return cudaSuccess;
}

// The call behind fm_attn_varlen and fm_attn_paged.
int attn_seqs(bool paged, const fm_tensor *q, const fm_tensor *k, const fm_tensor *v, const fm_seqs *seqs,
              const fm_seqs_opts *opts, const fm_tensor *o_out, float *lse, void *workspace, size_t workspace_bytes,
              fm_stream_t stream) {
  clear_error();
  SeqsArgs a;
  int rc;
  if ((rc = seqs_view(q, "q", &a.q)) || (rc = seqs_view(k, paged ? "k_cache" : "k", &a.k)) ||
      (rc = seqs_view(v, paged ? "v_cache" : "v", &a.v)) || (rc = seqs_view(o_out, "o_out", &a.o)))
    return rc;
  if (a.q.dtype != a.k.dtype || a.q.dtype != a.v.dtype) return fail(FM_ERR_DTYPE, "q, k and v must share one dtype");
  if (a.o.dtype != a.q.dtype && a.o.dtype != FM_F32) return fail(FM_ERR_DTYPE, "o_out must have q's dtype or be fp32");
  if (a.q.B != 1) return fail(FM_ERR_SHAPE, "q holds packed rows: its B must be 1 (got %lld)", (long long)a.q.B);
  if (!paged && a.k.B != 1) return fail(FM_ERR_SHAPE, "k holds packed rows: its B must be 1 (got %lld)", (long long)a.k.B);
  if (a.k.B != a.v.B || a.k.H != a.v.H || a.k.S != a.v.S) return fail(FM_ERR_SHAPE, "the shapes of k and v differ");
  if (a.k.D != a.q.D || a.v.D != a.q.D) return fail(FM_ERR_SHAPE, "head dimensions of q, k, v differ");
  if (a.o.B != 1 || a.o.H != a.q.H || a.o.S != a.q.S || a.o.D != a.q.D)
    return fail(FM_ERR_SHAPE, "o_out must have q's shape");
  if ((rc = check_group(a.q.H, a.k.H))) return rc;
  if (opts && ((opts->causal != 0 && opts->causal != 1) || opts->window < 0))
    return fail(FM_ERR_ARG, "causal must be 0 or 1 and window at least 0");
  a.causal = opts ? opts->causal : 1;
  a.window = opts ? opts->window : 0;
  if (a.window > 0 && !a.causal) return fail(FM_ERR_ARG, "a window needs causal = 1");
  if (a.window >= kMaxRows) a.window = 0;  // no request has more keys
  if (opts && isnan(opts->softmax_scale)) return fail(FM_ERR_ARG, "softmax_scale must be finite");
  const double scale = (opts && opts->softmax_scale > 0.f) ? (double)opts->softmax_scale : 1.0 / sqrt((double)a.q.D);
  a.alpha = (float)(scale * 1.4426950408889634);
  if (!isfinite(a.alpha)) return fail(FM_ERR_ARG, "softmax_scale must be finite, in base 2 (times log2 e) too");
  if (!seqs) return fail(FM_ERR_ARG, "seqs is NULL");
  a.paged = paged;
  a.n = seqs->n_seqs;
  if (a.n < 0) return fail(FM_ERR_ARG, "n_seqs = %lld", (long long)a.n);
  if (a.n > kMaxSeqs) return fail(FM_ERR_UNSUPPORTED, "%lld requests: at most %d", (long long)a.n, kMaxSeqs);
  if (a.n == 0 || a.q.S == 0) return FM_OK;
  a.cu_q = seqs->cu_q;
  a.cu_k = seqs->cu_k;
  a.kv_len = seqs->kv_len;
  a.table = seqs->block_table;
  a.table_stride = seqs->table_stride;
  a.table_width = seqs->table_width;
  if (!a.cu_q || misaligned(a.cu_q, 4)) return fail(FM_ERR_ARG, "cu_q must be given, 4-byte aligned");
  if (paged) {
    if (!a.kv_len || misaligned(a.kv_len, 4)) return fail(FM_ERR_ARG, "kv_len must be given, 4-byte aligned");
    if (a.k.S < 1 || a.k.S > INT_MAX) return fail(FM_ERR_SHAPE, "the cache's page size (its S) must be at least 1");
    if (a.table_width < 0 || a.table_width > INT_MAX || a.table_stride < 0 || (a.n > 1 && a.table_stride < a.table_width))
      return fail(FM_ERR_ARG, "block_table: rows of %lld entries %lld apart", (long long)a.table_width,
                  (long long)a.table_stride);
    if ((a.table_width > 0 && !a.table) || misaligned(a.table, 4))
      return fail(FM_ERR_ARG, "block_table must be given, 4-byte aligned");
  } else if (!a.cu_k || misaligned(a.cu_k, 4)) {
    return fail(FM_ERR_ARG, "cu_k must be given, 4-byte aligned");
  }
  if (misaligned(lse, 4)) return fail(FM_ERR_ARG, "lse must be 4-byte aligned");
  a.lse = lse;
  const int group = (int)(a.q.H / a.k.H);
  if ((a.q.S / (64 / group) + a.n) * a.k.H > kMaxRows)
    return fail(FM_ERR_UNSUPPORTED, "more than 2^30 units of work (query rows x heads)");
  const size_t need = space_bytes(a.n, a.q.S, a.q.H, a.k.H, a.q.D);
  if (workspace_bytes < need) return fail(FM_ERR_ARG, "workspace of %zu bytes < %zu needed", workspace_bytes, need);
  if (!workspace || misaligned(workspace, 16)) return fail(FM_ERR_ARG, "workspace must be given, 16-byte aligned");
  a.ws = reinterpret_cast<void *>((reinterpret_cast<uintptr_t>(workspace) + kSpaceAlign - 1) & ~(uintptr_t)(kSpaceAlign - 1));
  a.err = dev_error_ptr();
  a.timeout_ns = wait_timeout_ns();
  if (!a.err) return fail(FM_ERR_CUDA, "no CUDA device");
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = prepare();
  if (e != cudaSuccess) return cuda_fail(e, "preparing the attention kernels");
  // the work list, the attention, the merge of what was cut
  auto run = [&](const SeqsGeom &g, cudaError_t (*attend)(const SeqsArgs &, const SeqsGeom &, const SeqsSpace &, cudaStream_t)) {
    const SeqsSpace s = seqs_space(g, a.n, a.q.S, a.k.H, a.q.D);
    cudaError_t e = g.stream ? cudaSuccess : launch_seqs_plan(a, g, s, st);
    if (e == cudaSuccess) e = attend(a, g, s, st);
    if (e == cudaSuccess) e = launch_seqs_merge(a, g, s, st);
    return e;
  };
  e = cudaErrorNotSupported;
  if (seqs_tc_supported(a)) e = run(seqs_geom_tc(a.q.S, a.n, group), launch_seqs_tc);
  // fp32, and layouts that the tensor-core kernel or the tensor-map encoder does not take (a work
  // list made for it then goes unused)
  if (e == cudaErrorNotSupported)
    e = run(seqs_geom_simt(a.q.S, group, simt_rows(a.q.S, a.n, group)), launch_seqs_simt);
  if (e != cudaSuccess) return cuda_fail(e, paged ? "fm_attn_paged launch" : "fm_attn_varlen launch");
  return FM_OK;
}

}  // namespace

extern "C" {

int fm_attn_seqs_workspace_size(int64_t n_seqs, int64_t T, int64_t Hq, int64_t Hk, int64_t D, size_t *bytes) {
  clear_error();
  if (!bytes) return fail(FM_ERR_ARG, "bytes is NULL");
  if (n_seqs < 0 || T < 0 || D < 0) return fail(FM_ERR_ARG, "negative size");
  if (T > kMaxRows || n_seqs > kMaxSeqs) return fail(FM_ERR_UNSUPPORTED, "more than 2^30 rows or %d requests", kMaxSeqs);
  int rc;
  if ((rc = check_group(Hq, Hk))) return rc;
  *bytes = space_bytes(n_seqs, T, Hq, Hk, D);
  return FM_OK;
}

int fm_attn_varlen(const fm_tensor *q, const fm_tensor *k, const fm_tensor *v, const fm_seqs *seqs,
                   const fm_seqs_opts *opts, const fm_tensor *o_out, float *lse, void *workspace,
                   size_t workspace_bytes, fm_stream_t stream) {
  return attn_seqs(false, q, k, v, seqs, opts, o_out, lse, workspace, workspace_bytes, stream);
}

int fm_attn_paged(const fm_tensor *q, const fm_tensor *k_cache, const fm_tensor *v_cache, const fm_seqs *seqs,
                  const fm_seqs_opts *opts, const fm_tensor *o_out, float *lse, void *workspace,
                  size_t workspace_bytes, fm_stream_t stream) {
  return attn_seqs(true, q, k_cache, v_cache, seqs, opts, o_out, lse, workspace, workspace_bytes, stream);
}

int fm_paged_extend(const fm_page_state *state, const int32_t *new_len, const uint8_t *release, int64_t max_tokens,
                    int32_t *cu_q, int64_t *slots, int32_t *positions, int32_t *status, fm_stream_t stream) {
  clear_error();
  if (!state) return fail(FM_ERR_ARG, "state is NULL");
  const fm_page_state &s = *state;
  if (s.n_seqs < 0 || s.num_pages < 0 || s.table_width < 0 || s.table_stride < 0 || max_tokens < 0)
    return fail(FM_ERR_ARG, "negative size");
  if (s.page_size < 1) return fail(FM_ERR_ARG, "page_size = %lld", (long long)s.page_size);
  if (s.n_seqs > kMaxSeqs) return fail(FM_ERR_UNSUPPORTED, "%lld requests: at most %d", (long long)s.n_seqs, kMaxSeqs);
  if (s.page_size > kMaxRows || s.num_pages > kMaxRows || s.table_width > kMaxRows || max_tokens > kMaxRows)
    return fail(FM_ERR_UNSUPPORTED, "page size, pages, table width and tokens of a call are limited to 2^30");
  if (s.n_seqs > 1 && s.table_stride < s.table_width)
    return fail(FM_ERR_ARG, "block_table: rows of %lld entries %lld apart", (long long)s.table_width,
                (long long)s.table_stride);
  if (!cu_q || !status || !s.free_count || !s.free_count_out || (s.num_pages > 0 && !s.free_pages) ||
      (max_tokens > 0 && (!slots || !positions)) ||
      (s.n_seqs > 0 && (!new_len || !s.kv_len || !s.kv_len_out || (s.table_width > 0 && !s.block_table))))
    return fail(FM_ERR_ARG, "every array of fm_paged_extend but release must be given");
  if (misaligned(cu_q, 4) || misaligned(status, 4) || misaligned(s.free_count, 4) || misaligned(s.free_count_out, 4) ||
      misaligned(s.free_pages, 4) || misaligned(slots, 8) || misaligned(positions, 4) || misaligned(new_len, 4) ||
      misaligned(s.kv_len, 4) || misaligned(s.kv_len_out, 4) || misaligned(s.block_table, 4))
    return fail(FM_ERR_ARG, "the arrays of fm_paged_extend must be aligned to their elements");
  PagedExtendArgs a;
  a.n = s.n_seqs;
  a.page_size = s.page_size;
  a.num_pages = s.num_pages;
  a.table_stride = s.table_stride;
  a.table_width = s.table_width;
  a.max_tokens = max_tokens;
  a.new_len = new_len;
  a.release = release;
  a.kv_len = s.kv_len;
  a.kv_out = s.kv_len_out;
  a.table = s.block_table;
  a.free_pages = s.free_pages;
  a.free_count = s.free_count;
  a.free_out = s.free_count_out;
  a.cu_q = cu_q;
  a.slots = slots;
  a.positions = positions;
  a.status = status;
  const cudaError_t e = launch_paged_extend(a, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FM_OK : cuda_fail(e, "fm_paged_extend launch");
}

int fm_paged_write(const fm_tensor *k, const fm_tensor *v, const int64_t *slots, const fm_tensor *k_cache,
                   const fm_tensor *v_cache, fm_stream_t stream) {
  clear_error();
  View vk, vv, kc, vc;
  int rc;
  if ((rc = seqs_view(k, "k", &vk)) || (rc = seqs_view(v, "v", &vv)) || (rc = seqs_view(k_cache, "k_cache", &kc)) ||
      (rc = seqs_view(v_cache, "v_cache", &vc)))
    return rc;
  if (vk.dtype != vv.dtype || vk.dtype != kc.dtype || vk.dtype != vc.dtype)
    return fail(FM_ERR_DTYPE, "the rows and the caches must share one dtype");
  if (vk.B != 1 || vv.B != 1) return fail(FM_ERR_SHAPE, "k and v hold packed rows: their B must be 1");
  if (vk.S != vv.S || vk.H != vv.H || vk.D != vv.D) return fail(FM_ERR_SHAPE, "the shapes of k and v differ");
  if (kc.B != vc.B || kc.S != vc.S || kc.H != vk.H || vc.H != vk.H || kc.D != vk.D || vc.D != vk.D)
    return fail(FM_ERR_SHAPE, "the caches must be [pages, H, page size, D] with the rows' H and D");
  if (vk.S == 0 || vk.H == 0) return FM_OK;
  if (kc.S < 1) return fail(FM_ERR_SHAPE, "the cache's page size (its S) must be at least 1");
  if (!slots || misaligned(slots, 8)) return fail(FM_ERR_ARG, "slots must be given, 8-byte aligned");
  unsigned int *err = dev_error_ptr();
  if (!err) return fail(FM_ERR_CUDA, "no CUDA device");
  const cudaError_t e = launch_paged_write(vk, vv, slots, kc, vc, err, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FM_OK : cuda_fail(e, "fm_paged_write launch");
}

}  // extern "C"
