"""Host-side checks of the calls on trees of drafted tokens: every refusal happens before the device is touched (fake
device pointers are never dereferenced), and the binding refuses tensors that are not on the GPU."""
import ctypes
import os

import pytest
import torch

import fixed_max_softmax_gb300 as fm
from tests.test_seqs_cpu import FAKE, ROOT, lib, state, view  # noqa: F401


def tree(lib, q=None, k=None, o=None, opt=None, seqs=None, mask=FAKE, words=2, stride=2, nbytes=1 << 40):  # noqa: F811
    q, k = q or view(1, 8, 100, 128), k or view(40, 2, 16, 128)
    return lib.fm_attn_tree(ctypes.byref(q), ctypes.byref(k), ctypes.byref(k),
                            ctypes.byref(seqs or fm.fm_seqs(3, FAKE, None, FAKE, FAKE, 10, 10)), mask, words, stride,
                            ctypes.byref(opt or fm.seqs_opts()), ctypes.byref(o or q), None, FAKE, nbytes, None)


def test_tree_attention_refusals(lib):  # noqa: F811
    assert tree(lib, mask=None) == fm.FM_ERR_ARG and "mask" in fm.fm_last_error()
    assert tree(lib, mask=FAKE + 2) == fm.FM_ERR_ARG
    assert tree(lib, words=0) == fm.FM_ERR_ARG
    assert tree(lib, words=33, stride=33) == fm.FM_ERR_UNSUPPORTED
    assert tree(lib, words=2, stride=1) == fm.FM_ERR_ARG
    assert tree(lib, opt=fm.seqs_opts(causal=False)) == fm.FM_ERR_ARG
    assert tree(lib, opt=fm.seqs_opts(window=5)) == fm.FM_ERR_UNSUPPORTED
    assert tree(lib, q=view(1, 7, 100, 128)) == fm.FM_ERR_SHAPE
    assert tree(lib, q=view(1, 8, 100, 96), o=view(1, 8, 100, 96)) == fm.FM_ERR_UNSUPPORTED
    assert tree(lib, seqs=fm.fm_seqs(3, FAKE, None, None, FAKE, 10, 10)) == fm.FM_ERR_ARG
    assert tree(lib, nbytes=1000) == fm.FM_ERR_ARG and "workspace" in fm.fm_last_error()
    assert tree(lib, seqs=fm.fm_seqs(0, None, None, None, None, 0, 0)) == fm.FM_OK  # no request: nothing to do


def mask_call(lib, n=3, T=50, cu=FAKE, kv=FAKE, parent=FAKE, mask=FAKE, words=2, stride=2, pos=FAKE):  # noqa: F811
    return lib.fm_tree_mask(ctypes.byref(fm.fm_seqs(n, cu, None, kv, None, 0, 0)), parent, T, mask, words, stride, pos, None)


def test_mask_refusals(lib):  # noqa: F811
    assert lib.fm_tree_mask(None, FAKE, 1, FAKE, 1, 1, None, None) == fm.FM_ERR_ARG
    for kw in (dict(n=-1), dict(T=-1), dict(cu=None), dict(kv=None), dict(parent=None), dict(mask=None), dict(words=0),
               dict(stride=1), dict(cu=FAKE + 1), dict(kv=FAKE + 2), dict(parent=FAKE + 3), dict(mask=FAKE + 1), dict(pos=FAKE + 2)):
        assert mask_call(lib, **kw) == fm.FM_ERR_ARG, kw
    for kw in (dict(n=fm.FM_MAX_SEQS + 1), dict(T=2 ** 30 + 1), dict(words=33, stride=33)):
        assert mask_call(lib, **kw) == fm.FM_ERR_UNSUPPORTED, kw
    assert mask_call(lib, n=0) == fm.FM_OK and mask_call(lib, T=0, mask=None) == fm.FM_OK  # nothing to do


def test_constants_match_header():
    text = open(os.path.join(ROOT, "include", "fm.h")).read()
    assert f"#define FM_MAX_NODES {fm.FM_MAX_NODES} " in text


def test_binding_refusals(lib, monkeypatch):  # noqa: F811
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q, cache = torch.zeros(4, 2, 128, dtype=torch.bfloat16), torch.zeros(3, 2, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(fm.FMError, match="CUDA device"):
        fm.fm_attn_tree(q, cache, cache, i(2), i(1), i(1, 4), i(4, 1), fm.seqs_opts(), q)
    with pytest.raises(fm.FMError, match="CUDA device"):
        fm.fm_tree_mask(i(4), i(2), i(1), i(4, 1))
    for bad in (i(3, 1), i(4), i(1, 4).t().long(), torch.zeros(2, 4, dtype=torch.int32).t()):
        with pytest.raises(fm.FMError, match="mask must be"):
            fm._mask(bad, 4, -1)
    assert fm._mask(torch.zeros(4, 5, dtype=torch.int32)[:, 1:3], 4, -1)[1:] == (2, 5)


# ---------------------------------------------------------------- verification
def rows(T=50, V=1000, dtype=fm.FM_F32, ptr=FAKE, step=1):
    t = view(1, 1, T, V, dtype, ptr)
    t.stride[3] = step
    return t


def verify(lib, p=None, q=None, n=3, max_path=8, **kw):  # noqa: F811
    a = dict(cu=FAKE, tokens=FAKE, parent=FAKE, u=FAKE, u_last=FAKE, path=FAKE, kept=FAKE, nxt=FAKE)
    a.update(kw)
    return lib.fm_tree_verify(ctypes.byref(p or rows()), None if q is None else ctypes.byref(q), n, a["cu"], a["tokens"], a["parent"],
                              a["u"], a["u_last"], max_path, a["path"], a["kept"], a["nxt"], None)


def test_verify_refusals(lib):  # noqa: F811
    assert lib.fm_tree_verify(None, None, 1, FAKE, FAKE, FAKE, FAKE, FAKE, 1, FAKE, FAKE, FAKE, None) == fm.FM_ERR_ARG
    assert verify(lib, p=view(2, 1, 50, 1000, fm.FM_F32)) == fm.FM_ERR_SHAPE
    assert verify(lib, p=view(1, 2, 50, 1000, fm.FM_F32)) == fm.FM_ERR_SHAPE
    assert verify(lib, p=rows(V=0)) == fm.FM_ERR_ARG
    assert verify(lib, p=rows(ptr=None)) == fm.FM_ERR_ARG
    assert verify(lib, p=rows(ptr=FAKE + 2)) == fm.FM_ERR_UNSUPPORTED
    assert verify(lib, p=rows(step=2)) == fm.FM_ERR_UNSUPPORTED
    assert verify(lib, p=rows(V=2 ** 30 + 1)) == fm.FM_ERR_UNSUPPORTED
    assert verify(lib, p=rows(dtype=fm.FM_F8E4M3)) == fm.FM_ERR_DTYPE
    assert verify(lib, q=rows(dtype=fm.FM_BF16)) == fm.FM_ERR_DTYPE
    assert verify(lib, q=rows(T=49)) == fm.FM_ERR_SHAPE
    assert verify(lib, q=rows(V=999)) == fm.FM_ERR_SHAPE
    assert verify(lib, n=-1) == fm.FM_ERR_ARG
    assert verify(lib, n=fm.FM_MAX_SEQS + 1) == fm.FM_ERR_UNSUPPORTED
    assert verify(lib, max_path=0) == fm.FM_ERR_ARG
    assert verify(lib, max_path=fm.FM_MAX_NODES + 1) == fm.FM_ERR_UNSUPPORTED
    for name in ("cu", "tokens", "parent", "u", "u_last", "path", "kept", "nxt"):
        assert verify(lib, **{name: None}) == fm.FM_ERR_ARG, name
        assert verify(lib, **{name: FAKE + 2}) == fm.FM_ERR_ARG, name
    assert verify(lib, n=0, cu=None) == fm.FM_OK  # no request: nothing to do


def test_verify_binding_refusals(lib, monkeypatch):  # noqa: F811
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # (where get_device() says that host tensors are)
    i, f = (lambda *s: torch.zeros(s, dtype=torch.int32)), (lambda *s: torch.zeros(s))
    good = [f(4, 10), f(4, 10), i(3), i(4), i(4), f(4), f(2), i(2, 5), i(2), i(2)]
    for at, bad in ((0, f(4)), (2, i(3).long()), (3, i(3)), (4, i(4).long()), (5, i(4)), (6, f(1)), (7, i(10)), (7, i(1, 5)),
                    (7, i(5, 2).t()), (8, i(1)), (9, f(2))):
        with pytest.raises(fm.FMError):
            fm.fm_tree_verify(*good[:at], bad, *good[at + 1:], stream=0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(fm.FMError, match="CUDA device"):
        fm.fm_tree_verify(*good)


def test_the_definition_is_lossless():
    """Whatever the draft, the first new token is distributed as the target's row: children drawn from q, each kept or
    refused by the definition, summed over every way that it can go, in exact fractions."""
    from fractions import Fraction as F
    p, q = [F(1, 2), F(1, 8), F(3, 8), F(0)], [F(1, 8), F(1, 2), F(1, 4), F(1, 8)]
    for children in (0, 1, 2, 3):
        got = [F(0)] * 4

        def go(weight, a, mass, left_children):
            left = [max(x - a * y, F(0)) for x, y in zip(p, q)]
            if left_children == 0:
                total = sum(left)
                for x in range(4):
                    got[x] += weight * left[x] / total
                return
            refused = F(0)
            for x in range(4):  # the child's token, drawn from q; kept where u q S < what is left of p
                keep = min(F(1), left[x] / (q[x] * mass))
                got[x] += weight * q[x] * keep
                refused += q[x] * (1 - keep)
            if refused:
                nxt = a + mass
                rest = sum(max(x - nxt * y, F(0)) for x, y in zip(p, q))
                go(weight * refused, *((nxt, rest) if rest else (F(0), F(1))), left_children - 1)

        go(F(1), F(0), F(1), children)
        assert got == p, children


# ---------------------------------------------------------------- what is kept
def keep(lib, st, width=4, cu=FAKE, path=FAKE, kept=FAKE, src=FAKE, dst=FAKE, status=FAKE):  # noqa: F811
    return lib.fm_paged_keep(ctypes.byref(st), cu, width, path, kept, src, dst, status, None)


def test_keep_refusals(lib):  # noqa: F811
    assert lib.fm_paged_keep(None, FAKE, 1, FAKE, FAKE, FAKE, FAKE, FAKE, None) == fm.FM_ERR_ARG
    for kw in (dict(n_seqs=-1), dict(page_size=0), dict(num_pages=-1), dict(table_width=-1), dict(table_stride=7), dict(free_pages=None),
               dict(free_count=None), dict(free_count_out=None), dict(kv_len=None), dict(kv_len_out=None), dict(block_table=None),
               dict(kv_len=FAKE + 2)):
        assert keep(lib, state(**kw)) == fm.FM_ERR_ARG, kw
    assert keep(lib, state(n_seqs=fm.FM_MAX_SEQS + 1)) == fm.FM_ERR_UNSUPPORTED
    assert keep(lib, state(), width=fm.FM_MAX_NODES + 1) == fm.FM_ERR_UNSUPPORTED
    for kw in (dict(width=0), dict(cu=None), dict(path=None), dict(kept=None), dict(src=None), dict(dst=None), dict(status=None),
               dict(src=FAKE + 4), dict(dst=FAKE + 4), dict(cu=FAKE + 1), dict(path=FAKE + 2), dict(kept=FAKE + 3), dict(status=FAKE + 1)):
        assert keep(lib, state(), **kw) == fm.FM_ERR_ARG, kw


def test_move_refusals(lib):  # noqa: F811
    def move(kc=None, vc=None, n=3, width=4, src=FAKE, dst=FAKE):
        kc = kc or view(9, 2, 16, 128)
        return lib.fm_paged_move(n, width, src, dst, ctypes.byref(kc), ctypes.byref(vc or kc), None)
    assert move(vc=view(9, 2, 32, 128)) == fm.FM_ERR_SHAPE
    assert move(vc=view(9, 2, 16, 128, fm.FM_F16)) == fm.FM_ERR_DTYPE
    assert move(kc=view(9, 2, 16, 96)) == fm.FM_ERR_UNSUPPORTED
    assert move(kc=view(9, 2, 0, 128)) == fm.FM_ERR_SHAPE
    assert move(n=-1) == fm.FM_ERR_ARG and move(width=-1) == fm.FM_ERR_ARG
    assert move(n=fm.FM_MAX_SEQS + 1) == fm.FM_ERR_UNSUPPORTED and move(width=fm.FM_MAX_NODES + 1) == fm.FM_ERR_UNSUPPORTED
    for bad in (None, FAKE + 4):
        assert move(src=bad) == fm.FM_ERR_ARG and move(dst=bad) == fm.FM_ERR_ARG
    assert move(n=0, src=None) == fm.FM_OK and move(width=0, src=None) == fm.FM_OK  # nothing to do


def test_keep_and_move_binding_refusals(lib, monkeypatch):  # noqa: F811
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # (where get_device() says that host tensors are)
    i, w = (lambda *s: torch.zeros(s, dtype=torch.int32)), (lambda *s: torch.zeros(s, dtype=torch.int64))
    good = [i(3), i(2, 5), i(2), i(2), i(2), i(2, 4), i(8), i(1), i(1), 16, w(2, 5), w(2, 5), i(1)]
    for at, bad in ((0, i(2)), (1, i(10)), (1, i(1, 5)), (1, i(5, 2).t()), (1, w(2, 5)), (2, i(4)[::2]), (3, i(1)), (4, w(2)), (5, i(8)),
                    (6, w(8)), (7, i(0)), (8, i(0)), (10, i(2, 5)), (11, w(9)), (12, i(0))):
        with pytest.raises(fm.FMError):
            fm.fm_paged_keep(*good[:at], bad, *good[at + 1:], stream=0)
    cache = torch.zeros(3, 2, 16, 128)
    for src, dst in ((w(2, 5), w(2, 4)), (w(10), w(10)), (i(2, 5), w(2, 5)), (w(5, 2).t(), w(2, 5))):
        with pytest.raises(fm.FMError):
            fm.fm_paged_move(src, dst, cache, cache, stream=0)
    c = fm.PagedKVCache(6, 4, 2, 64, 3, 5, 7, device="cpu")
    with pytest.raises(fm.FMError, match="each of the 3 rows"):
        c.keep(i(2, 4), i(2))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(fm.FMError, match="CUDA device"):
        fm.fm_paged_keep(*good)
    with pytest.raises(fm.FMError, match="CUDA device"):
        fm.fm_paged_move(w(2, 5), w(2, 5), cache, cache)


def test_moves_are_of_the_caches_rows_alone(monkeypatch):
    """A path buffer with more rows than the cache: fm_paged_keep fills the moves of the cache's, so that there are no
    others for fm_paged_move to make."""
    c, got = fm.PagedKVCache(6, 4, 2, 64, 3, 5, 7, device="cpu"), {}
    monkeypatch.setattr(fm, "fm_paged_keep", lambda *a, **kw: got.update(src=a[10], dst=a[11]))
    for rows in (3, 9):
        moves = c.keep(torch.zeros(rows, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
        assert moves.shape == (2, 3, 2) and got["src"].shape == got["dst"].shape == (3, 2)
    monkeypatch.undo()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # (where get_device() says that host tensors are)
    for bad in (torch.zeros(6, dtype=torch.int32), torch.zeros(2, 2, dtype=torch.int32), torch.zeros((), dtype=torch.int32)):
        with pytest.raises(fm.FMError, match="path must be"):
            c.keep(bad, torch.zeros(3, dtype=torch.int32))


def test_keep_has_a_status_of_its_own(monkeypatch):
    """What extend reported stays until the next one; layers that share tables share both."""
    c = fm.PagedKVCache(6, 4, 2, 64, 3, 5, 7, device="cpu")
    other = fm.PagedKVCache(6, 4, 2, 64, 3, 5, 7, device="cpu", shared=c)
    monkeypatch.setattr(fm, "fm_paged_keep", lambda *a, **kw: a[12].fill_(2))
    c.status.fill_(5)
    c.keep(torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
    for x in (c, other):
        assert x.status.tolist() == [5] and x.keep_status.tolist() == [2]


# ---------------------------------------------------------------- verification of steps that are not all trees
def verify_rows(lib, p=None, n=3, T=70, max_path=8, **kw):  # noqa: F811
    a = dict(cu=FAKE, rows=FAKE, tokens=FAKE, parent=FAKE, u=FAKE, u_last=FAKE, path=FAKE, kept=FAKE, nxt=FAKE)
    a.update(kw)
    return lib.fm_tree_verify_rows(ctypes.byref(p or rows()), None, n, a["cu"], a["rows"], T, a["tokens"], a["parent"], a["u"],
                                   a["u_last"], max_path, a["path"], a["kept"], a["nxt"], None)


def test_verify_rows_refusals(lib):  # noqa: F811
    for name in ("cu", "rows", "tokens", "parent", "u", "u_last", "path", "kept", "nxt"):
        assert verify_rows(lib, **{name: None}) == fm.FM_ERR_ARG, name
        assert verify_rows(lib, **{name: FAKE + 2}) == fm.FM_ERR_ARG, name
    assert verify_rows(lib, T=-1) == fm.FM_ERR_ARG and verify_rows(lib, n=-1) == fm.FM_ERR_ARG
    assert verify_rows(lib, T=2 ** 30 + 1) == fm.FM_ERR_UNSUPPORTED
    assert verify_rows(lib, n=fm.FM_MAX_SEQS + 1) == fm.FM_ERR_UNSUPPORTED
    assert verify_rows(lib, max_path=0) == fm.FM_ERR_ARG and verify_rows(lib, p=rows(step=2)) == fm.FM_ERR_UNSUPPORTED
    assert verify_rows(lib, p=view(1, 2, 50, 1000, fm.FM_F32)) == fm.FM_ERR_SHAPE
    assert verify_rows(lib, n=0, cu=None, rows=None) == fm.FM_OK  # no request: nothing to do


def test_verify_rows_binding_refusals(lib, monkeypatch):  # noqa: F811
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # (where get_device() says that host tensors are)
    i, f = (lambda *s: torch.zeros(s, dtype=torch.int32)), (lambda *s: torch.zeros(s))
    good = [f(4, 10), f(4, 10), i(3), i(9), i(9), f(9), f(2), i(2, 5), i(2), i(2)]
    for bad in (i(1), i(2).long(), f(2), i(4)[::2]):
        with pytest.raises(fm.FMError, match="rows"):
            fm.fm_tree_verify(*good, stream=0, rows=bad)
    for at, bad in ((4, i(8)), (5, f(8)), (3, i(9).long()), (8, i(1))):
        with pytest.raises(fm.FMError):
            fm.fm_tree_verify(*good[:at], bad, *good[at + 1:], stream=0, rows=i(2))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(fm.FMError, match="CUDA device"):
        fm.fm_tree_verify(*good, rows=i(2))
