"""Host-side checks of the calls on trees of drafted tokens: every refusal happens before the device is touched (fake
device pointers are never dereferenced), and the binding refuses tensors that are not on the GPU."""
import ctypes
import os

import pytest
import torch

import fixed_max_softmax_gb300 as fm
from tests.test_seqs_cpu import FAKE, ROOT, lib, view  # noqa: F401


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
