"""fixed_max_softmax_gb300 -- fixed-m (const-max) attention forward on GB300.

A thin ctypes binding of ``libfm.so`` (C ABI: ``include/fm.h``).  Every step of the
path -- bounds, chunk folding, finalize -- runs in the library's CUDA kernels; this
module only marshals torch tensors into ``fm_tensor`` descriptors, passes raw
pointers and the current CUDA stream, and turns error codes into exceptions.
PyTorch provides device memory and streams and nothing else.

Functions with the ABI's names (same arguments, torch tensors in place of pointers):
``fm_bounds_workspace_size``, ``fm_bounds``, ``fm_bounds_noalloc``, ``fm_attn_chunk``,
``fm_attn_chunk_final``, ``fm_attn_chunks``, ``fm_fold_sinks``, ``fm_finalize``,
``fm_finalize_lse``, ``fm_sync_status``,
``fm_probe_wait_timeout``,
``fm_last_error``, ``fm_version``; and for requests of different lengths
``fm_attn_seqs_workspace_size``, ``fm_attn_varlen``, ``fm_attn_paged``, ``fm_paged_extend``,
``fm_paged_write``; for trees of drafted tokens ``fm_tree_mask``, ``fm_attn_tree``, ``fm_tree_verify``,
``fm_tree_verify_rows``, ``fm_paged_keep``, ``fm_paged_move``.

``FixedMAttention`` owns the buffers of one problem shape and runs the whole path
(bounds, one ``fm_attn_chunk`` per KV chunk, finalize); ``attention()`` is the
one-call form.  ``attention_varlen()`` is the one-call form of packed prompts, ``PagedKVCache``
owns a paged cache with its bookkeeping (extend, write, attention; for drafted tokens tree,
tree_attention, keep, move), ``verify_tree()`` is the one-call form of the verification.

There is no CPU path: if the library is not built, ``load()`` raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libfm.so")
DEBUG_LIB_PATH = os.path.join(_HERE, "_build_debug", "libfm.so")  # build(debug=True): kernel index checks

FM_F32, FM_BF16, FM_F16, FM_F8E4M3, FM_F8E5M2 = 0, 1, 2, 3, 4
FM_OK, FM_ERR_ARG, FM_ERR_SHAPE, FM_ERR_DTYPE, FM_ERR_UNSUPPORTED = 0, 1, 2, 3, 4
FM_ERR_BOUNDS_MISMATCH, FM_ERR_CUDA, FM_ERR_TIMEOUT, FM_ERR_INDEX = 5, 6, 7, 8
FM_BOUNDS_MAGIC = 0x314D4246
FM_BOUNDS_LOCAL_MAGIC = 0x314C4246
FM_BLOCK_Q = 128
ERROR_NAMES = {0: "FM_OK", 1: "FM_ERR_ARG", 2: "FM_ERR_SHAPE", 3: "FM_ERR_DTYPE", 4: "FM_ERR_UNSUPPORTED",
               5: "FM_ERR_BOUNDS_MISMATCH", 6: "FM_ERR_CUDA", 7: "FM_ERR_TIMEOUT", 8: "FM_ERR_INDEX"}
ABI_SYMBOLS = ("fm_bounds_workspace_size", "fm_bounds", "fm_attn_chunk", "fm_finalize", "fm_sync_status",
               "fm_last_error", "fm_version", "fm_bounds_noalloc", "fm_finalize_lse", "fm_probe_wait_timeout",
               "fm_attn_chunk_final", "fm_attn_chunks", "fm_fold_sinks", "fm_ring_stats_bytes", "fm_ring_key_sums",
               "fm_bounds_local", "fm_bounds_combine", "fm_attention_host", "fm_attn_seqs_workspace_size",
               "fm_attn_varlen", "fm_attn_paged", "fm_paged_extend", "fm_paged_write", "fm_tree_mask", "fm_attn_tree",
               "fm_tree_verify", "fm_tree_verify_rows", "fm_paged_keep", "fm_paged_move")
FM_MAX_CHUNKS = 8
FM_MAX_SINKS = 8
FM_NOALLOC_SCRATCH_BYTES = 4 << 20
FM_MAX_GROUP = 64
FM_MAX_SEQS = 8192
FM_MAX_NODES = 1024


class FMError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{ERROR_NAMES.get(code, code)}: {msg}")
        self.code = code


class fm_tensor(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("B", ctypes.c_int64), ("H", ctypes.c_int64), ("S", ctypes.c_int64), ("D", ctypes.c_int64),
                ("stride", ctypes.c_int64 * 4)]


class fm_opts(ctypes.Structure):
    _fields_ = [("softmax_scale", ctypes.c_float), ("centering", ctypes.c_int32),
                ("force_online", ctypes.c_int32), ("per_row", ctypes.c_int32), ("sink_keys", ctypes.c_int32),
                ("schedule", ctypes.c_int32)]


class fm_bounds_out(ctypes.Structure):
    _fields_ = [("m", ctypes.c_void_p), ("flag", ctypes.c_void_p), ("qmax_sq", ctypes.c_void_p),
                ("kmax_sq", ctypes.c_void_p), ("kbar", ctypes.c_void_p), ("qkbar", ctypes.c_void_p),
                ("shift", ctypes.c_void_p), ("vmax_sq", ctypes.c_void_p),
                ("sink_idx", ctypes.c_void_p), ("sink_k", ctypes.c_void_p), ("sink_v", ctypes.c_void_p),
                ("B", ctypes.c_int64), ("H", ctypes.c_int64), ("Sq", ctypes.c_int64), ("D", ctypes.c_int64),
                ("n_qblocks", ctypes.c_int64), ("N_total", ctypes.c_int64),
                ("C", ctypes.c_int32), ("W", ctypes.c_int32), ("gate", ctypes.c_int32),
                ("centered", ctypes.c_int32), ("per_row", ctypes.c_int32), ("n_sink", ctypes.c_int32),
                ("alpha", ctypes.c_float), ("dtype", ctypes.c_int32),
                ("kv_seen", ctypes.c_int64), ("next_key_offset", ctypes.c_int64), ("online_lock", ctypes.c_int32),
                ("sinks_folded", ctypes.c_int32),
                ("magic", ctypes.c_uint32)]


class fm_host_buffers(ctypes.Structure):
    _fields_ = [("q", fm_tensor * 2), ("k", fm_tensor * 2), ("v", fm_tensor * 2), ("o", fm_tensor * 2),
                ("acc_o", ctypes.c_void_p), ("acc_sum", ctypes.c_void_p), ("acc_max", ctypes.c_void_p),
                ("bounds", ctypes.POINTER(fm_bounds_out)), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


class fm_seqs_opts(ctypes.Structure):
    _fields_ = [("softmax_scale", ctypes.c_float), ("causal", ctypes.c_int32), ("window", ctypes.c_int32)]


class fm_seqs(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int64), ("cu_q", ctypes.c_void_p), ("cu_k", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("table_width", ctypes.c_int64)]


class fm_page_state(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int64), ("page_size", ctypes.c_int64), ("num_pages", ctypes.c_int64),
                ("block_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("table_width", ctypes.c_int64),
                ("free_pages", ctypes.c_void_p), ("free_count", ctypes.c_void_p), ("free_count_out", ctypes.c_void_p),
                ("kv_len", ctypes.c_void_p), ("kv_len_out", ctypes.c_void_p)]


_lib = None


def load(path: str | None = None):
    """Load libfm.so (build it first with fixed_max_softmax_gb300.build.build())."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise FMError(FM_ERR_CUDA, f"{p} is missing: the CUDA library is not built "
                                   "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(p)
    P, i64 = ctypes.c_void_p, ctypes.c_int64
    lib.fm_bounds_workspace_size.argtypes = [i64, i64, i64, i64, ctypes.POINTER(ctypes.c_size_t)]
    lib.fm_bounds.argtypes = [P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.fm_attn_chunk.argtypes = [P, P, P, P, P, P, P, P, ctypes.c_int, P]
    lib.fm_finalize.argtypes = [P, P, P, P]
    lib.fm_bounds_noalloc.argtypes = [P, P, P, P, P, P]
    lib.fm_finalize_lse.argtypes = [P, P, P, P, P, P]
    lib.fm_probe_wait_timeout.argtypes = [ctypes.c_uint, P]
    lib.fm_attn_chunk_final.argtypes = [P, P, P, P, P, P, P, P, ctypes.c_int, P, P, P]
    lib.fm_attn_chunks.argtypes = [P, P, P, ctypes.c_int, P, P, P, P, P, ctypes.c_int, P, P, P]
    lib.fm_fold_sinks.argtypes = [P, P, P, P, P, P, P]
    lib.fm_ring_stats_bytes.argtypes = [i64, i64, i64, ctypes.c_int, ctypes.POINTER(ctypes.c_size_t)]
    lib.fm_ring_key_sums.argtypes = [P, P, P, ctypes.c_size_t, P]
    lib.fm_bounds_local.argtypes = [P, P, P, i64, i64, P, P, P, P, P, ctypes.c_size_t, P]
    lib.fm_bounds_combine.argtypes = [P, ctypes.c_int, P, P, P]
    lib.fm_attention_host.argtypes = [P, P, P, P, ctypes.c_int, P, ctypes.c_int, P, P, P]
    lib.fm_attn_seqs_workspace_size.argtypes = [i64, i64, i64, i64, i64, ctypes.POINTER(ctypes.c_size_t)]
    lib.fm_attn_varlen.argtypes = [P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.fm_attn_paged.argtypes = [P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.fm_paged_extend.argtypes = [P, P, P, i64, P, P, P, P, P]
    lib.fm_paged_write.argtypes = [P, P, P, P, P, P]
    lib.fm_tree_mask.argtypes = [P, P, i64, P, i64, i64, P, P]
    lib.fm_attn_tree.argtypes = [P, P, P, P, P, i64, i64, P, P, P, P, ctypes.c_size_t, P]
    lib.fm_tree_verify.argtypes = [P, P, i64, P, P, P, P, P, i64, P, P, P, P]
    lib.fm_tree_verify_rows.argtypes = [P, P, i64, P, P, i64, P, P, P, P, i64, P, P, P, P]
    lib.fm_paged_keep.argtypes = [P, P, i64, P, P, P, P, P, P]
    lib.fm_paged_move.argtypes = [i64, i64, P, P, P, P, P]
    lib.fm_sync_status.argtypes = [P]
    lib.fm_last_error.restype = ctypes.c_char_p
    lib.fm_last_error.argtypes = []
    lib.fm_version.argtypes = []
    for name in ("fm_bounds_workspace_size", "fm_bounds", "fm_attn_chunk", "fm_finalize", "fm_sync_status",
                 "fm_version", "fm_bounds_noalloc", "fm_finalize_lse", "fm_probe_wait_timeout",
                 "fm_attn_chunk_final", "fm_attn_chunks", "fm_fold_sinks", "fm_ring_stats_bytes", "fm_ring_key_sums",
                 "fm_bounds_local", "fm_bounds_combine", "fm_attention_host", "fm_attn_seqs_workspace_size",
                 "fm_attn_varlen", "fm_attn_paged", "fm_paged_extend", "fm_paged_write", "fm_tree_mask", "fm_attn_tree",
                 "fm_tree_verify", "fm_tree_verify_rows", "fm_paged_keep", "fm_paged_move"):
        getattr(lib, name).restype = ctypes.c_int
    _lib = lib
    return lib


_DTYPES = {torch.float32: FM_F32, torch.bfloat16: FM_BF16, torch.float16: FM_F16}
if hasattr(torch, "float8_e4m3fn"):
    _DTYPES[torch.float8_e4m3fn] = FM_F8E4M3
if hasattr(torch, "float8_e5m2"):
    _DTYPES[torch.float8_e5m2] = FM_F8E5M2


def tensor(t: torch.Tensor) -> fm_tensor:
    """Describe a 4-D [B, H, S, D] torch tensor (any strides) as an fm_tensor."""
    if t.dim() != 4:
        raise FMError(FM_ERR_SHAPE, f"expected a 4-D [B, H, S, D] tensor, got shape {tuple(t.shape)}")
    d = fm_tensor()
    d.ptr = t.data_ptr() or None
    d.dtype = _DTYPES.get(t.dtype, -1)
    d.B, d.H, d.S, d.D = t.shape
    for i, s in enumerate(t.stride()):
        d.stride[i] = s
    return d


FM_SCHEDULE_AUTO, FM_SCHEDULE_GRID, FM_SCHEDULE_PERSISTENT = 0, 1, 2
SCHEDULES = {"auto": FM_SCHEDULE_AUTO, "grid": FM_SCHEDULE_GRID, "persistent": FM_SCHEDULE_PERSISTENT}


def opts(softmax_scale: float = 0.0, centering: bool = False, force_online: bool = False,
         per_row: bool = False, sink_keys: int = 0, schedule="auto") -> fm_opts:
    sched = SCHEDULES[schedule] if isinstance(schedule, str) else int(schedule)
    return fm_opts(float(softmax_scale), int(bool(centering)), int(bool(force_online)), int(bool(per_row)),
                   int(sink_keys), sched)


def _stream(stream):
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(rc: int):
    if rc != FM_OK:
        raise FMError(rc, load().fm_last_error().decode())
    return rc


def fm_version() -> int:
    return load().fm_version()


def fm_last_error() -> str:
    return load().fm_last_error().decode()


def fm_bounds_workspace_size(B: int, H: int, N_total: int, D: int) -> int:
    n = ctypes.c_size_t()
    _check(load().fm_bounds_workspace_size(B, H, N_total, D, ctypes.byref(n)))
    return n.value


class Bounds:
    """Device arrays of one fm_bounds_out (allocated with torch) plus the struct itself."""

    def __init__(self, B: int, H: int, Sq: int, D: int, device):
        nqb = (Sq + FM_BLOCK_Q - 1) // FM_BLOCK_Q
        kw = dict(device=device)
        self.m = torch.zeros(B, H, nqb, dtype=torch.int32, **kw)
        self.flag = torch.zeros(B, H, nqb, dtype=torch.uint8, **kw)
        self.qmax_sq = torch.zeros(B, H, nqb, dtype=torch.float32, **kw)
        self.kmax_sq = torch.zeros(B, H, dtype=torch.float32, **kw)
        self.kbar = torch.zeros(B, H, D, dtype=torch.float32, **kw)
        self.qkbar = torch.zeros(B, H, max(Sq, 1), dtype=torch.float32, **kw)
        self.shift = torch.zeros(B, H, max(Sq, 1), dtype=torch.float32, **kw)
        self.vmax_sq = torch.zeros(1, dtype=torch.float32, **kw)
        self.sink_idx = torch.zeros(B, H, FM_MAX_SINKS, dtype=torch.int32, **kw)
        self.sink_k = torch.zeros(B, H, FM_MAX_SINKS, D, dtype=torch.float32, **kw)
        self.sink_v = torch.zeros(B, H, FM_MAX_SINKS, D, dtype=torch.float32, **kw)
        self.out = fm_bounds_out()
        self.out.m, self.out.flag = self.m.data_ptr(), self.flag.data_ptr()
        self.out.qmax_sq, self.out.kmax_sq = self.qmax_sq.data_ptr(), self.kmax_sq.data_ptr()
        self.out.kbar, self.out.qkbar, self.out.vmax_sq = (self.kbar.data_ptr(), self.qkbar.data_ptr(),
                                                           self.vmax_sq.data_ptr())
        self.out.shift = self.shift.data_ptr()
        self.out.sink_idx, self.out.sink_k, self.out.sink_v = (self.sink_idx.data_ptr(), self.sink_k.data_ptr(),
                                                               self.sink_v.data_ptr())


def fm_bounds(q, k_full, v_full, opt: fm_opts, bounds: Bounds, workspace: torch.Tensor | None, stream=None):
    tq, tk, tv = tensor(q), tensor(k_full), tensor(v_full)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return _check(load().fm_bounds(ctypes.byref(tq), ctypes.byref(tk), ctypes.byref(tv), ctypes.byref(opt),
                                   ctypes.byref(bounds.out), _ptr(workspace), ws_bytes, _stream(stream)))


def fm_bounds_noalloc(q, k_full, v_full, opt: fm_opts, bounds: Bounds, stream=None):
    """fm_bounds without a workspace: the library's static device scratch is used instead
    (for callers that cannot allocate; see include/fm.h)."""
    tq, tk, tv = tensor(q), tensor(k_full), tensor(v_full)
    return _check(load().fm_bounds_noalloc(ctypes.byref(tq), ctypes.byref(tk), ctypes.byref(tv), ctypes.byref(opt),
                                           ctypes.byref(bounds.out), _stream(stream)))


def fm_ring_stats_bytes(B: int, H: int, D: int, sink_keys: int = 0) -> int:
    n = ctypes.c_size_t()
    _check(load().fm_ring_stats_bytes(B, H, D, int(sink_keys), ctypes.byref(n)))
    return n.value


def fm_ring_key_sums(k_shard, ksum, workspace, stream=None):
    """ksum [B, H, D] f32 <- the sums of this rank's keys (step 1 of the ring bounds)."""
    tk = tensor(k_shard)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return _check(load().fm_ring_key_sums(ctypes.byref(tk), _ptr(ksum), _ptr(workspace), ws_bytes, _stream(stream)))


def fm_bounds_local(q, k_shard, v_shard, key_offset: int, N_total: int, ksum_total, opt: fm_opts, bounds: Bounds,
                    stats, workspace, stream=None):
    """This rank's part of the bounds: bounds' query-side arrays and its statistics block (step 2)."""
    tq, tk, tv = tensor(q), tensor(k_shard), tensor(v_shard)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return _check(load().fm_bounds_local(ctypes.byref(tq), ctypes.byref(tk), ctypes.byref(tv), int(key_offset),
                                         int(N_total), _ptr(ksum_total), ctypes.byref(opt), ctypes.byref(bounds.out),
                                         _ptr(stats), _ptr(workspace), ws_bytes, _stream(stream)))


def fm_bounds_combine(stats_all, n_ranks: int, opt: fm_opts, bounds: Bounds, stream=None):
    """Every rank's statistics blocks (rank order) -> the rest of the bounds (step 3)."""
    return _check(load().fm_bounds_combine(_ptr(stats_all), int(n_ranks), ctypes.byref(opt), ctypes.byref(bounds.out),
                                           _stream(stream)))


def fm_attn_chunk(q, k_chunk, v_chunk, bounds: Bounds, opt: fm_opts, acc_o, acc_sum, acc_max,
                  accumulate: bool, stream=None):
    tq, tk, tv = tensor(q), tensor(k_chunk), tensor(v_chunk)
    return _check(load().fm_attn_chunk(ctypes.byref(tq), ctypes.byref(tk), ctypes.byref(tv),
                                       ctypes.byref(bounds.out), ctypes.byref(opt), _ptr(acc_o), _ptr(acc_sum),
                                       _ptr(acc_max), int(bool(accumulate)), _stream(stream)))


def fm_attn_chunk_final(q, k_chunk, v_chunk, bounds: Bounds, opt: fm_opts, acc_o, acc_sum, acc_max,
                        accumulate: bool, o_out, lse=None, stream=None):
    tq, tk, tv, to = tensor(q), tensor(k_chunk), tensor(v_chunk), tensor(o_out)
    return _check(load().fm_attn_chunk_final(ctypes.byref(tq), ctypes.byref(tk), ctypes.byref(tv),
                                             ctypes.byref(bounds.out), ctypes.byref(opt), _ptr(acc_o),
                                             _ptr(acc_sum), _ptr(acc_max), int(bool(accumulate)), ctypes.byref(to),
                                             _ptr(lse), _stream(stream)))


def fm_attn_chunks(q, k_chunks, v_chunks, bounds: Bounds, opt: fm_opts, acc_o, acc_sum, acc_max,
                   accumulate: bool, o_out=None, lse=None, stream=None):
    """Fold a list of consecutive KV chunks in one pass (and normalise into o_out if given)."""
    n = len(k_chunks)
    ks = (fm_tensor * n)(*[tensor(t) for t in k_chunks])
    vs = (fm_tensor * n)(*[tensor(t) for t in v_chunks])
    to = tensor(o_out) if o_out is not None else None
    return _check(load().fm_attn_chunks(ctypes.byref(tensor(q)), ks, vs, n, ctypes.byref(bounds.out),
                                        ctypes.byref(opt), _ptr(acc_o), _ptr(acc_sum), _ptr(acc_max),
                                        int(bool(accumulate)), None if to is None else ctypes.byref(to), _ptr(lse),
                                        _stream(stream)))


def fm_fold_sinks(q, bounds: Bounds, opt: fm_opts, acc_o, acc_sum, acc_max, stream=None):
    """Merge the key sinks set aside by fm_bounds back into the accumulators (after the last
    chunk, before fm_finalize); a no-op without sinks."""
    tq = tensor(q)
    return _check(load().fm_fold_sinks(ctypes.byref(tq), ctypes.byref(bounds.out), ctypes.byref(opt), _ptr(acc_o),
                                       _ptr(acc_sum), _ptr(acc_max), _stream(stream)))


def fm_finalize(acc_o, acc_sum, o_out, stream=None):
    to = tensor(o_out)
    return _check(load().fm_finalize(_ptr(acc_o), _ptr(acc_sum), ctypes.byref(to), _stream(stream)))


def fm_finalize_lse(acc_o, acc_sum, acc_max, o_out, lse, stream=None):
    to = tensor(o_out)
    return _check(load().fm_finalize_lse(_ptr(acc_o), _ptr(acc_sum), _ptr(acc_max), ctypes.byref(to), _ptr(lse),
                                         _stream(stream)))


def fm_sync_status(stream=None):
    return _check(load().fm_sync_status(_stream(stream)))


def fm_probe_wait_timeout(timeout_ms: int, stream=None):
    return _check(load().fm_probe_wait_timeout(int(timeout_ms), _stream(stream)))


class FixedMAttention:
    """Buffers and the call sequence of one fixed-m attention forward of a fixed shape.

    forward(q, k, v, chunks) runs fm_bounds over all of K/V, one fm_attn_chunk per
    (start, length) slice of the key sequence (the ring's steps, sequentially) and writes
    `out` (fp32 or the input dtype): by default the last chunk goes through
    fm_attn_chunk_final (fold and normalise in one pass); fused_final=False uses a separate
    fm_finalize.  one_launch=True folds all chunks with fm_attn_chunks instead (one launch per
    FM_MAX_CHUNKS chunks, accumulators on chip across them).  with_lse=True also fills
    `lse` [B, H, Sq] (natural log).  sink_keys > 0 leaves that many of each head's loudest
    keys out of the key max; they are folded back exactly before the normalise.  schedule:
    "auto", "grid" or "persistent" (fm_opts.schedule; the same bits either way).
    """

    def __init__(self, B, H, Sq, N, D, device="cuda", centering=False, softmax_scale=0.0,
                 force_online=False, out_dtype=torch.float32, per_row=False, sink_keys=0, schedule="auto"):
        self.shape = (B, H, Sq, N, D)
        self.opt = opts(softmax_scale, centering, force_online, per_row, sink_keys, schedule)
        self.bounds = Bounds(B, H, Sq, D, device)
        nbytes = fm_bounds_workspace_size(B, H, N, D)
        self.workspace = torch.empty(max(nbytes, 16) // 4 + 4, dtype=torch.float32, device=device)
        self.acc_o = torch.empty(B, H, Sq, D, dtype=torch.float32, device=device)
        self.acc_sum = torch.empty(B, H, Sq, dtype=torch.float32, device=device)
        self.acc_max = torch.empty(B, H, Sq, dtype=torch.float32, device=device)
        self.out = torch.empty(B, H, Sq, D, dtype=out_dtype, device=device)
        self.lse = None

    def forward(self, q, k, v, chunks=None, stream=None, with_lse=False, fused_final=True, one_launch=False):
        N = k.shape[2]
        chunks = [(0, N)] if chunks is None else chunks
        fm_bounds(q, k, v, self.opt, self.bounds, self.workspace, stream)
        if with_lse and self.lse is None:
            self.lse = torch.empty(self.acc_sum.shape, dtype=torch.float32, device=self.acc_sum.device)
        lse = self.lse if with_lse else None
        if one_launch:  # every chunk (up to FM_MAX_CHUNKS per call) and the normalise in one pass
            for g0 in range(0, len(chunks), FM_MAX_CHUNKS):
                grp = chunks[g0:g0 + FM_MAX_CHUNKS]
                last = g0 + FM_MAX_CHUNKS >= len(chunks)
                if any(grp[i][0] + grp[i][1] != grp[i + 1][0] for i in range(len(grp) - 1)):
                    raise ValueError("one_launch folds consecutive key ranges only")
                self.bounds.out.next_key_offset = grp[0][0]
                fm_attn_chunks(q, [k[:, :, s:s + n] for s, n in grp], [v[:, :, s:s + n] for s, n in grp],
                               self.bounds, self.opt, self.acc_o, self.acc_sum, self.acc_max, g0 > 0,
                               self.out if last else None, lse if last else None, stream)
            return self.out
        for i, (s, n) in enumerate(chunks):
            kc, vc = k[:, :, s:s + n], v[:, :, s:s + n]
            self.bounds.out.next_key_offset = s  # the chunk's global key offset: any order works
            if fused_final and i == len(chunks) - 1:
                fm_attn_chunk_final(q, kc, vc, self.bounds, self.opt, self.acc_o, self.acc_sum, self.acc_max, i > 0,
                                    self.out, lse, stream)
                return self.out
            fm_attn_chunk(q, kc, vc, self.bounds, self.opt, self.acc_o, self.acc_sum, self.acc_max, i > 0, stream)
        fm_fold_sinks(q, self.bounds, self.opt, self.acc_o, self.acc_sum, self.acc_max, stream)
        if with_lse:
            fm_finalize_lse(self.acc_o, self.acc_sum, self.acc_max, self.out, self.lse, stream)
        else:
            fm_finalize(self.acc_o, self.acc_sum, self.out, stream)
        return self.out

    __call__ = forward


def attention(q, k, v, chunks=None, centering=False, softmax_scale=0.0, force_online=False,
              out_dtype=torch.float32, stream=None, per_row=False, sink_keys=0):
    """One-call fixed-m attention forward: returns o [B, H, Sq, D]."""
    B, H, Sq, D = q.shape
    fa = FixedMAttention(B, H, Sq, k.shape[2], D, q.device, centering, softmax_scale, force_online, out_dtype,
                         per_row, sink_keys)
    return fa.forward(q, k, v, chunks, stream).clone()


class HostPipeline:
    """Fixed-m attention over a stream of batches that live in (pinned) host memory, through
    fm_attention_host: batch i+1's inputs are copied to the device on one stream while batch i
    computes on another, and batch i-1's output is read back on a third.  Every batch still makes
    the full host -> device -> host round trip, but the copies hide behind the kernels.  Two
    device copies of the inputs and of the output alternate between batches; the bounds,
    accumulators and workspace of `fa` are reused in order.
    """

    def __init__(self, fa: FixedMAttention, in_dtype, device="cuda"):
        B, H, Sq, N, D = fa.shape
        self.fa = fa
        self.device = torch.device(device)
        self.q = [torch.empty(B, H, Sq, D, dtype=in_dtype, device=device) for _ in range(2)]
        self.k = [torch.empty(B, H, N, D, dtype=in_dtype, device=device) for _ in range(2)]
        self.v = [torch.empty(B, H, N, D, dtype=in_dtype, device=device) for _ in range(2)]
        self.o = [torch.empty_like(fa.out) for _ in range(2)]
        self.streams = [torch.cuda.Stream(device=device) for _ in range(3)]
        self.dev = fm_host_buffers()
        for i in range(2):
            self.dev.q[i], self.dev.k[i], self.dev.v[i], self.dev.o[i] = (tensor(self.q[i]), tensor(self.k[i]),
                                                                          tensor(self.v[i]), tensor(self.o[i]))
        self.dev.acc_o, self.dev.acc_sum, self.dev.acc_max = (fa.acc_o.data_ptr(), fa.acc_sum.data_ptr(),
                                                              fa.acc_max.data_ptr())
        self.dev.bounds = ctypes.pointer(fa.bounds.out)
        self.dev.workspace = fa.workspace.data_ptr()
        self.dev.workspace_bytes = fa.workspace.numel() * fa.workspace.element_size()

    def run(self, batches, chunks=None):
        """batches: a list of (q_host, k_host, v_host, o_host); o_host is filled.  chunks: the
        (start, length) key ranges, consecutive from 0.  Returns when every output is back in
        host memory."""
        batches = list(batches)
        N = self.k[0].shape[2]
        chunks = [(0, N)] if chunks is None else chunks
        if [s for s, _ in chunks] != [sum(n for _, n in chunks[:i]) for i in range(len(chunks))]:
            raise ValueError("chunks must be consecutive key ranges from 0")
        n = len(batches)
        qs = (fm_tensor * max(n, 1))(*[tensor(b[0]) for b in batches])
        ks = (fm_tensor * max(n, 1))(*[tensor(b[1]) for b in batches])
        vs = (fm_tensor * max(n, 1))(*[tensor(b[2]) for b in batches])
        os_ = (fm_tensor * max(n, 1))(*[tensor(b[3]) for b in batches])
        lens = (ctypes.c_int64 * len(chunks))(*[c for _, c in chunks])
        st = (ctypes.c_void_p * 3)(*[s.cuda_stream for s in self.streams])
        return _check(load().fm_attention_host(qs, ks, vs, os_, n, lens, len(chunks), ctypes.byref(self.fa.opt),
                                               ctypes.byref(self.dev), st))


# ---- requests of different lengths, and a paged key/value cache ------------------------------------
def seqs_opts(causal: bool = True, window: int = 0, softmax_scale: float = 0.0) -> fm_seqs_opts:
    # (a C int32 would take the window's low 32 bits; no request has 2^31 keys)
    return fm_seqs_opts(float(softmax_scale), int(bool(causal)), max(-1, min(int(window), 2 ** 31 - 1)))


# These calls are made once a layer and step, often for a few microseconds of work, so their arguments
# go to the library as packed bytes (the layouts of fm_tensor, fm_seqs and fm_page_state).
_TENSOR_BYTES, _SEQS_BYTES, _STATE_BYTES = struct.Struct("=Qii8q").pack, struct.Struct("=q4Q2q").pack, struct.Struct("=3qQ2q5Q").pack


def _rows(t: torch.Tensor, name: str, device: int) -> bytes:
    """fm_tensor of packed rows: a [T, H, D] tensor, or a [1, H, T, D] one (any strides)."""
    if t.dim() == 4:
        return _cache(t, name, device)
    if t.dim() != 3:
        raise FMError(FM_ERR_SHAPE, f"{name}: expected a [T, H, D] or [1, H, T, D] tensor, got shape {tuple(t.shape)}")
    if t.get_device() != device:
        _not_here(t, name, device)
    (S, H, D), (sS, sH, sD) = t.shape, t.stride()
    return _TENSOR_BYTES(t.data_ptr(), _DTYPES.get(t.dtype, -1), 0, 1, H, S, D, 0, sH, sS, sD)


def _cache(t: torch.Tensor, name: str, device: int) -> bytes:
    """fm_tensor of a 4-D [B, H, S, D] tensor (any strides)."""
    if t.dim() != 4:
        raise FMError(FM_ERR_SHAPE, f"{name}: expected a 4-D tensor, got shape {tuple(t.shape)}")
    if t.get_device() != device:
        _not_here(t, name, device)
    return _TENSOR_BYTES(t.data_ptr(), _DTYPES.get(t.dtype, -1), 0, *t.shape, *t.stride())


def _not_here(t, name, device):
    """The kernels get raw pointers: every tensor has to be on the current device."""
    raise FMError(FM_ERR_ARG, f"{name} must be on the current CUDA device (cuda:{device}), not {t.device}")


def _ints(t, dtype, numel, name, device):
    """Data pointer of a contiguous tensor of that dtype and of at least numel elements."""
    if t.dtype != dtype or not t.is_contiguous() or t.numel() < numel:
        raise FMError(FM_ERR_ARG, f"{name} must be a contiguous {dtype} tensor of at least {numel} elements, got "
                                  f"{tuple(t.shape)} {t.dtype}")
    if t.get_device() != device:
        _not_here(t, name, device)
    return t.data_ptr()


def _table(t, n, device):
    (rows, width), (stride, step) = (t.shape, t.stride()) if t.dim() == 2 else ((-2, 0), (0, 0))
    if rows < n or t.dtype != torch.int32 or (width > 1 and step != 1):
        raise FMError(FM_ERR_ARG, f"block_table must be a 2-D int32 tensor of at least {n} rows with adjacent "
                                  f"entries, got {tuple(t.shape)} {t.dtype}")
    if t.get_device() != device:
        _not_here(t, "block_table", device)
    return t.data_ptr(), stride, width


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the handle alone: a tenth of the time


def _stream_handle(stream, device):
    if stream is None:
        return _raw_stream(device) if _raw_stream else torch.cuda.current_stream(device).cuda_stream
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def fm_attn_seqs_workspace_size(n_seqs: int, T: int, Hq: int, Hk: int, D: int) -> int:
    n = ctypes.c_size_t()
    _check(load().fm_attn_seqs_workspace_size(n_seqs, T, Hq, Hk, D, ctypes.byref(n)))
    return n.value


def _attn_seqs(fn, q, k, v, seqs, opt, o_out, lse, workspace, stream, device, mask=()):
    if lse is not None:
        heads, rows = (q.shape[1], q.shape[0]) if q.dim() == 3 else (q.shape[1], q.shape[2])
        if lse.dtype != torch.float32 or not lse.is_contiguous() or lse.numel() != heads * rows:
            raise FMError(FM_ERR_ARG, f"lse must be a contiguous float32 [{heads}, {rows}] tensor, got {tuple(lse.shape)}")
        if lse.get_device() != device:
            _not_here(lse, "lse", device)
        lse = lse.data_ptr()
    ws = nbytes = 0
    if workspace is not None:
        if not workspace.is_contiguous():  # its elements' bytes would not be a range that the kernels may write
            raise FMError(FM_ERR_ARG, f"workspace must be contiguous, got shape {tuple(workspace.shape)}, strides {workspace.stride()}")
        if workspace.get_device() != device:
            _not_here(workspace, "workspace", device)
        ws, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    rc = fn(_rows(q, "q", device), k, v, seqs, *mask, ctypes.byref(opt), _rows(o_out, "o_out", device), lse, ws, nbytes,
            _stream_handle(stream, device))
    return rc if rc == FM_OK else _check(rc)


def fm_attn_varlen(q, k, v, cu_q, cu_k, opt: fm_seqs_opts, o_out, lse=None, workspace=None, stream=None):
    """Attention of packed requests: q, o_out [T, Hq, D], k, v [Tk, Hk, D] (or [1, H, T, D]); request i
    owns rows cu[i] .. cu[i+1]-1 of each.  lse [Hq, T]; see include/fm.h."""
    dev, n, i32 = torch.cuda.current_device(), cu_q.numel() - 1, torch.int32
    seqs = _SEQS_BYTES(n, _ints(cu_q, i32, 1, "cu_q", dev), _ints(cu_k, i32, n + 1, "cu_k", dev), 0, 0, 0, 0)
    return _attn_seqs(load().fm_attn_varlen, q, _rows(k, "k", dev), _rows(v, "v", dev), seqs, opt, o_out, lse, workspace,
                      stream, dev)


def fm_attn_paged(q, k_cache, v_cache, cu_q, kv_len, block_table, opt: fm_seqs_opts, o_out, lse=None, workspace=None,
                  stream=None):
    """Attention of each request's new tokens (q, o_out [T, Hq, D], packed by cu_q) over its pages:
    caches [pages, Hk, page_size, D] (any strides), block_table int32 [n, width], kv_len int32 [n]
    with the new tokens counted; see include/fm.h."""
    dev, n, i32 = torch.cuda.current_device(), cu_q.numel() - 1, torch.int32
    table, stride, width = _table(block_table, n, dev)
    seqs = _SEQS_BYTES(n, _ints(cu_q, i32, 1, "cu_q", dev), 0, _ints(kv_len, i32, n, "kv_len", dev), table, stride, width)
    return _attn_seqs(load().fm_attn_paged, q, _cache(k_cache, "k_cache", dev), _cache(v_cache, "v_cache", dev), seqs, opt,
                      o_out, lse, workspace, stream, dev)


def _mask(t, rows, device):
    """Data pointer, words and stride of a tree mask: a row for each of `rows` tokens."""
    (have, words), (stride, step) = (t.shape, t.stride()) if t.dim() == 2 else ((-2, 0), (0, 0))
    if have < rows or t.dtype != torch.int32 or (words > 1 and step != 1):
        raise FMError(FM_ERR_ARG, f"mask must be a 2-D int32 tensor of at least {rows} rows with adjacent words, got "
                                  f"{tuple(t.shape)} {t.dtype}")
    if t.get_device() != device:
        _not_here(t, "mask", device)
    return t.data_ptr(), words, stride


def fm_tree_mask(parent, cu_q, kv_len, mask, positions=None, stream=None):
    """mask int32 [T, words] (bit j of word j / 32) and positions int32 [T] of trees of drafted tokens: parent
    int32 [T] counts from each request's first node, -1 a root; see include/fm.h."""
    dev, n, i32, T = torch.cuda.current_device(), cu_q.numel() - 1, torch.int32, parent.numel()
    seqs = _SEQS_BYTES(n, _ints(cu_q, i32, 1, "cu_q", dev), 0, _ints(kv_len, i32, n, "kv_len", dev), 0, 0, 0)
    rc = load().fm_tree_mask(seqs, _ints(parent, i32, 0, "parent", dev), T, *_mask(mask, T, dev),
                             None if positions is None else _ints(positions, i32, T, "positions", dev),
                             _stream_handle(stream, dev))
    return rc if rc == FM_OK else _check(rc)


def fm_attn_tree(q, k_cache, v_cache, cu_q, kv_len, block_table, mask, opt: fm_seqs_opts, o_out, lse=None, workspace=None,
                 stream=None):
    """fm_attn_paged where of its request's new tokens each row sees those that its row of mask (int32
    [T, words], from fm_tree_mask) names; see include/fm.h."""
    dev, n, i32 = torch.cuda.current_device(), cu_q.numel() - 1, torch.int32
    table, stride, width = _table(block_table, n, dev)
    seqs = _SEQS_BYTES(n, _ints(cu_q, i32, 1, "cu_q", dev), 0, _ints(kv_len, i32, n, "kv_len", dev), table, stride, width)
    rows = q.shape[0] if q.dim() == 3 else q.shape[2] if q.dim() == 4 else 0
    return _attn_seqs(load().fm_attn_tree, q, _cache(k_cache, "k_cache", dev), _cache(v_cache, "v_cache", dev), seqs, opt,
                      o_out, lse, workspace, stream, dev, _mask(mask, rows, dev))


def _probabilities(t, name, device):
    """fm_tensor of a [T, V] tensor."""
    if t.dim() != 2:
        raise FMError(FM_ERR_SHAPE, f"{name}: expected a [T, V] tensor, got shape {tuple(t.shape)}")
    if t.get_device() != device:
        _not_here(t, name, device)
    (T, V), (sT, sV) = t.shape, t.stride()
    return _TENSOR_BYTES(t.data_ptr(), _DTYPES.get(t.dtype, -1), 0, 1, 1, T, V, 0, 0, sT, sV)


def fm_tree_verify(target, draft, cu_q, tokens, parent, u, u_last, path, kept, next_token, stream=None, rows=None):
    """target and draft [T, V] probabilities after each node (draft None: the nodes were chosen, not drawn);
    tokens, parent int32 [T], u float32 [T], u_last [n]; fills path int32 [n, max_path], kept and
    next_token int32 [n].  rows int32 [n] (fm_tree_verify_rows): the row of target and draft after each request's
    node 0, which then need rows for nodes alone; -1: a request that is no tree (a prompt chunk of any length) is
    passed over, its kept -1; see include/fm.h."""
    dev, n, i32, f32 = torch.cuda.current_device(), cu_q.numel() - 1, torch.int32, torch.float32
    T = target.shape[0] if rows is None else tokens.numel()
    if path.dim() != 2 or path.shape[0] < n:
        raise FMError(FM_ERR_ARG, f"path must be a contiguous int32 [{n}, max_path] tensor, got {tuple(path.shape)}")
    fn, at = (load().fm_tree_verify, ()) if rows is None else (load().fm_tree_verify_rows, (_ints(rows, i32, n, "rows", dev), T))
    rc = fn(_probabilities(target, "target", dev), None if draft is None else _probabilities(draft, "draft", dev),
            n, _ints(cu_q, i32, 1, "cu_q", dev), *at, _ints(tokens, i32, T, "tokens", dev),
            _ints(parent, i32, T, "parent", dev), _ints(u, f32, T, "u", dev), _ints(u_last, f32, n, "u_last", dev),
            path.shape[1], _ints(path, i32, 0, "path", dev), _ints(kept, i32, n, "kept", dev),
            _ints(next_token, i32, n, "next_token", dev), _stream_handle(stream, dev))
    return rc if rc == FM_OK else _check(rc)


def fm_paged_extend(new_len, release, kv_len, kv_len_out, block_table, free_pages, free_count, free_count_out,
                    page_size: int, cu_q, slots, positions, status, stream=None):
    """Room in the pages for new_len[i] more tokens of every request (release[i] != 0: the row's
    request has ended and gives its pages back first).  kv_len_out and free_count_out may be kv_len
    and free_count.  Fills cu_q [n+1], slots and positions [max tokens], status [1]; see include/fm.h."""
    dev, n, cap, i32 = torch.cuda.current_device(), new_len.numel(), slots.numel(), torch.int32
    table, stride, width = _table(block_table, n, dev)
    st = _STATE_BYTES(n, page_size, free_pages.numel(), table, stride, width,
                      _ints(free_pages, i32, 0, "free_pages", dev), _ints(free_count, i32, 1, "free_count", dev),
                      _ints(free_count_out, i32, 1, "free_count_out", dev), _ints(kv_len, i32, n, "kv_len", dev),
                      _ints(kv_len_out, i32, n, "kv_len_out", dev))
    rc = load().fm_paged_extend(st, _ints(new_len, i32, n, "new_len", dev),
                                None if release is None else _ints(release, torch.uint8, n, "release", dev), cap,
                                _ints(cu_q, i32, n + 1, "cu_q", dev), _ints(slots, torch.int64, cap, "slots", dev),
                                _ints(positions, i32, cap, "positions", dev), _ints(status, i32, 1, "status", dev),
                                _stream_handle(stream, dev))
    return rc if rc == FM_OK else _check(rc)


def fm_paged_write(k, v, slots, k_cache, v_cache, stream=None):
    """k, v rows [T, H, D] (or [1, H, T, D]) put at their slots of the caches [pages, H, page_size, D]."""
    dev = torch.cuda.current_device()
    rows = k.shape[0] if k.dim() == 3 else k.shape[2]
    rc = load().fm_paged_write(_rows(k, "k", dev), _rows(v, "v", dev), _ints(slots, torch.int64, rows, "slots", dev),
                               _cache(k_cache, "k_cache", dev), _cache(v_cache, "v_cache", dev), _stream_handle(stream, dev))
    return rc if rc == FM_OK else _check(rc)


def fm_paged_keep(cu_q, path, kept, kv_len, kv_len_out, block_table, free_pages, free_count, free_count_out, page_size: int,
                  src, dst, status, stream=None):
    """Of each request's new tokens only the first kept[i] of path[i] stay (-1: all): lengths, pages back to the list,
    and the moves src, dst int64 [n, max_path] that fm_paged_move makes in each layer (of larger buffers the first
    n * max_path are filled, and only they are moves); see include/fm.h."""
    dev, n, i32, i64 = torch.cuda.current_device(), kept.numel(), torch.int32, torch.int64
    if path.dim() != 2 or path.shape[0] < n:
        raise FMError(FM_ERR_ARG, f"path must be a contiguous int32 [{n}, max_path] tensor, got {tuple(path.shape)}")
    width = path.shape[1]
    table, stride, cols = _table(block_table, n, dev)
    st = _STATE_BYTES(n, page_size, free_pages.numel(), table, stride, cols,
                      _ints(free_pages, i32, 0, "free_pages", dev), _ints(free_count, i32, 1, "free_count", dev),
                      _ints(free_count_out, i32, 1, "free_count_out", dev), _ints(kv_len, i32, n, "kv_len", dev),
                      _ints(kv_len_out, i32, n, "kv_len_out", dev))
    rc = load().fm_paged_keep(st, _ints(cu_q, i32, n + 1, "cu_q", dev), width, _ints(path, i32, 0, "path", dev),
                              _ints(kept, i32, n, "kept", dev), _ints(src, i64, n * width, "src", dev),
                              _ints(dst, i64, n * width, "dst", dev), _ints(status, i32, 1, "status", dev),
                              _stream_handle(stream, dev))
    return rc if rc == FM_OK else _check(rc)


def fm_paged_move(src, dst, k_cache, v_cache, stream=None):
    """One layer's rows moved: src, dst int64 [n, max_path] from fm_paged_keep."""
    dev = torch.cuda.current_device()
    if src.dim() != 2 or src.shape != dst.shape:
        raise FMError(FM_ERR_SHAPE, f"src and dst must be [n, max_path] tensors, got {tuple(src.shape)} and {tuple(dst.shape)}")
    rc = load().fm_paged_move(src.shape[0], src.shape[1], _ints(src, torch.int64, 0, "src", dev),
                              _ints(dst, torch.int64, 0, "dst", dev), _cache(k_cache, "k_cache", dev),
                              _cache(v_cache, "v_cache", dev), _stream_handle(stream, dev))
    return rc if rc == FM_OK else _check(rc)


def _on_stream(stream):
    """Context whose current stream is `stream` (None: as it is), so that what it allocates belongs to it."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream)))


def attention_varlen(q, k, v, cu_q, cu_k=None, causal=True, window=0, softmax_scale=0.0, out_dtype=None, with_lse=False,
                     stream=None):
    """One-call attention of packed requests: returns o [T, Hq, D] (and lse [Hq, T]).  q [T, Hq, D],
    k, v [Tk, Hk, D], cu_q and cu_k int32 [n+1] (cu_k None: the same as cu_q)."""
    T, Hq, D = q.shape
    with _on_stream(stream):
        o = torch.zeros(T, Hq, D, dtype=out_dtype or q.dtype, device=q.device)  # rows behind the last request stay zero
        lse = torch.full((Hq, T), float("-inf"), dtype=torch.float32, device=q.device) if with_lse else None
        ws = torch.empty(fm_attn_seqs_workspace_size(cu_q.numel() - 1, T, Hq, k.shape[1], D), dtype=torch.uint8,
                         device=q.device)
        fm_attn_varlen(q, k, v, cu_q, cu_q if cu_k is None else cu_k, seqs_opts(causal, window, softmax_scale), o, lse, ws)
    return (o, lse) if with_lse else o


def verify_tree(target, tokens, parent, cu_q, u, u_last, draft=None, max_path=16, stream=None, rows=None):
    """One-call verification of trees of drafted tokens (fm_tree_verify): returns path int32 [n, max_path], kept and
    next_token int32 [n].  In a step with prompt chunks beside trees, rows int32 [n] says which row of target and draft
    comes after each tree's node 0, -1 for a chunk: it needs no rows, and its kept is -1, with which
    PagedKVCache.keep leaves all its tokens."""
    with _on_stream(stream):
        n, make = cu_q.numel() - 1, lambda *shape: torch.empty(shape, dtype=torch.int32, device=target.device)
        path, kept, next_token = make(n, max_path), make(n), make(n)
        fm_tree_verify(target, draft, cu_q, tokens, parent, u, u_last, path, kept, next_token, rows=rows)
    return path, kept, next_token


class PagedKVCache:
    """A paged key/value cache of one layer and the bookkeeping of up to max_seqs requests.

    extend(new_len, release) makes room for the next tokens and fills cu_q, slots, positions and
    kv_len; write(k, v) puts their rows into the pages; attention(q) attends over them.  Everything
    stays on the device: nothing here waits for the GPU, and status (0: the last extend fitted) is read
    when the caller chooses.  Several layers share one bookkeeping by sharing it: PagedKVCache(...,
    shared=first) keeps pages of its own (heads, head dimension and type as it likes) and uses the first
    layer's tables, so that its num_pages, page_size and limits have to be the first one's.

    New tokens may be drafted trees: after extend, mask = tree(parent) says what each node sees and sets
    positions by depth, tree_attention(q, mask) takes attention's place, and when verify_tree() has told
    what is kept, moves = keep(path, kept) cuts the lengths back and each layer's move(moves) puts the
    kept rows in their places, before the next extend.  A step whose extend did not fit has no new tokens, keeps none,
    and its status stays until the next extend; keep_status (0: every path could be) is keep's own."""

    def __init__(self, num_pages, page_size, kv_heads, head_dim, max_seqs, max_pages_per_seq, max_tokens,
                 dtype=torch.bfloat16, device="cuda", shared: "PagedKVCache | None" = None):
        make = lambda *shape: torch.zeros(shape, dtype=torch.int32, device=device)  # noqa: E731
        self.page_size = int(page_size)
        pages = torch.empty(2, num_pages, page_size, kv_heads, head_dim, dtype=dtype, device=device)
        self.k, self.v = pages[0].transpose(1, 2), pages[1].transpose(1, 2)  # [pages, heads, page_size, D]
        if shared is not None:
            if (shared.page_size, shared.free_pages.numel()) != (self.page_size, num_pages):
                raise FMError(FM_ERR_SHAPE, "layers that share tables need the same pages")
            has = (shared.kv_len.numel(), shared.block_table.shape[1], shared.slots.numel())
            if has != (max_seqs, max_pages_per_seq, max_tokens):
                raise FMError(FM_ERR_SHAPE, "layers that share tables have the first one's max_seqs, max_pages_per_seq and "
                                            f"max_tokens {has}, not {(max_seqs, max_pages_per_seq, max_tokens)}")
            if shared.kv_len.device != pages.device:
                raise FMError(FM_ERR_ARG, f"layers that share tables are on one device: {shared.kv_len.device}, not {pages.device}")
            for name in ("block_table", "free_pages", "free_count", "kv_len", "cu_q", "slots", "positions", "status", "keep_status"):
                setattr(self, name, getattr(shared, name))
        else:
            self.block_table = make(max_seqs, max_pages_per_seq)
            self.free_pages = torch.arange(num_pages - 1, -1, -1, dtype=torch.int32, device=device)
            self.free_count = make(1).fill_(num_pages)
            self.kv_len, self.cu_q, self.status, self.keep_status = make(max_seqs), make(max_seqs + 1), make(1), make(1)
            self.slots = torch.full((max_tokens,), -1, dtype=torch.int64, device=device)
            self.positions = make(max_tokens).fill_(-1)

    def extend(self, new_len, release=None, stream=None):
        """new_len int32 [max_seqs] (0: no new token in that row), release uint8 [max_seqs] or None."""
        if new_len.numel() != self.kv_len.numel():
            raise FMError(FM_ERR_SHAPE, f"new_len must have one entry for each of the {self.kv_len.numel()} rows")
        fm_paged_extend(new_len, release, self.kv_len, self.kv_len, self.block_table, self.free_pages, self.free_count,
                        self.free_count, self.page_size, self.cu_q, self.slots, self.positions, self.status, stream)

    def write(self, k, v, stream=None):
        """k, v [T, H, D], T <= max_tokens: the rows of the last extend, in its order (rows behind its
        last token are skipped)."""
        fm_paged_write(k, v, self.slots, self.k, self.v, stream)

    def attention(self, q, out=None, lse=None, causal=True, window=0, softmax_scale=0.0, stream=None):
        """q [T, Hq, D], the new tokens' queries in the order of the last extend; returns o [T, Hq, D]
        (rows behind the last token are left as they were in `out`, zero without one).  A step that is
        not captured is quicker with `out`: nothing has to be filled with zeros."""
        T, Hq, D = q.shape
        with _on_stream(stream):
            if out is None:
                out = torch.zeros(T, Hq, D, dtype=q.dtype, device=q.device)
            # from the allocator each time: a captured graph keeps its own, and no two calls share one
            ws = torch.empty(fm_attn_seqs_workspace_size(self.kv_len.numel(), T, Hq, self.k.shape[1], D),
                             dtype=torch.uint8, device=q.device)
            fm_attn_paged(q, self.k, self.v, self.cu_q, self.kv_len, self.block_table,
                          seqs_opts(causal, window, softmax_scale), out, lse, ws)
        return out

    def tree(self, parent, words=None, stream=None):
        """parent int32 [T]: each new token's parent among its request's new tokens, -1 for a root.  Returns the mask int32
        [T, words] (words: of 32 nodes, by default enough for T nodes in one tree, at most 32); positions become those of
        the nodes' depths.  A request of more than 32 * words new tokens (a prompt chunk) is causal; a shorter chunk is
        where each of its tokens has the one before it as its parent."""
        T = parent.numel()
        words = max(1, min(FM_MAX_NODES, T + 31) // 32) if words is None else words
        with _on_stream(stream):
            mask = torch.zeros(T, words, dtype=torch.int32, device=parent.device)  # rows behind the last token stay zero
            fm_tree_mask(parent, self.cu_q, self.kv_len, mask, self.positions)
        return mask

    def tree_attention(self, q, mask, out=None, lse=None, softmax_scale=0.0, stream=None):
        """As attention, of new tokens that see their request's earlier ones as mask says."""
        T, Hq, D = q.shape
        with _on_stream(stream):
            if out is None:
                out = torch.zeros(T, Hq, D, dtype=q.dtype, device=q.device)
            ws = torch.empty(fm_attn_seqs_workspace_size(self.kv_len.numel(), T, Hq, self.k.shape[1], D),
                             dtype=torch.uint8, device=q.device)
            fm_attn_tree(q, self.k, self.v, self.cu_q, self.kv_len, self.block_table, mask, seqs_opts(softmax_scale=softmax_scale),
                         out, lse, ws)
        return out

    def keep(self, path, kept, stream=None):
        """path int32 [max_seqs, max_path], kept int32 [max_seqs] from verify_tree (kept -1: a row keeps all its new
        tokens).  Returns the moves that move() makes in each layer; keep_status (of this call, as status is of extend)
        counts the rows whose path could not be."""
        if kept.numel() != self.kv_len.numel():
            raise FMError(FM_ERR_SHAPE, f"kept must have one entry for each of the {self.kv_len.numel()} rows")
        with _on_stream(stream):
            # (path may be the buffer of a larger batch: only the cache's rows have moves)
            moves = torch.empty(2, kept.numel(), *path.shape[1:], dtype=torch.int64, device=path.device)
            fm_paged_keep(self.cu_q, path, kept, self.kv_len, self.kv_len, self.block_table, self.free_pages, self.free_count,
                          self.free_count, self.page_size, moves[0], moves[1], self.keep_status)
        return moves

    def move(self, moves, stream=None):
        """This layer's rows of the tokens kept, put in their places."""
        fm_paged_move(moves[0], moves[1], self.k, self.v, stream)
