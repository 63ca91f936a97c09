"""Host-side checks of the calls over requests of different lengths and the paged cache: every
refusal happens before the device is touched (fake device pointers are never dereferenced), and the
binding refuses tensors that are not on the GPU."""
import ctypes
import os
import subprocess

import pytest
import torch

import fixed_max_softmax_gb300 as fm
from fixed_max_softmax_gb300 import build as fmbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    fmbuild.build()
    return fm.load()


def view(B, H, S, D, dtype=fm.FM_BF16, ptr=FAKE):
    t = fm.fm_tensor(ptr, dtype, 0, B, H, S, D)
    for i, s in enumerate((H * S * D, S * D, D, 1)):
        t.stride[i] = s
    return t


def attn(lib, paged=False, q=None, k=None, v=None, o=None, opt=None, seqs=None, ws=FAKE, nbytes=1 << 40, lse=None):
    q = q or view(1, 8, 100, 128)
    k = k or (view(40, 2, 16, 128) if paged else view(1, 2, 300, 128))
    v = v or k
    o = o or q
    seqs = seqs or fm.fm_seqs(3, FAKE, FAKE, FAKE, FAKE, 10, 10)
    fn = lib.fm_attn_paged if paged else lib.fm_attn_varlen
    return fn(ctypes.byref(q), ctypes.byref(k), ctypes.byref(v), ctypes.byref(seqs), ctypes.byref(opt or fm.seqs_opts()),
              ctypes.byref(o), lse, ws, nbytes, None)


@pytest.mark.parametrize("paged", [False, True])
def test_attention_refusals(lib, paged):
    r = lambda **kw: attn(lib, paged, **kw)  # noqa: E731
    assert r(q=view(1, 8, 100, 96), o=view(1, 8, 100, 96)) == fm.FM_ERR_UNSUPPORTED
    assert r(q=view(2, 8, 100, 128)) == fm.FM_ERR_SHAPE
    assert r(q=view(1, 7, 100, 128)) == fm.FM_ERR_SHAPE                      # 7 heads over 2
    assert r(q=view(1, 2 * 65, 100, 128)) == fm.FM_ERR_UNSUPPORTED           # 65 heads to one
    assert r(q=view(1, 8, 100, 128, fm.FM_F16)) == fm.FM_ERR_DTYPE           # mixed types
    assert r(q=view(1, 8, 100, 128, fm.FM_F8E4M3)) == fm.FM_ERR_DTYPE
    assert r(o=view(1, 8, 99, 128)) == fm.FM_ERR_SHAPE
    assert r(o=view(1, 8, 100, 128, fm.FM_F16)) == fm.FM_ERR_DTYPE
    assert r(v=view(40, 2, 32, 128) if paged else view(1, 2, 301, 128)) == fm.FM_ERR_SHAPE
    assert r(opt=fm.seqs_opts(causal=False, window=5)) == fm.FM_ERR_ARG
    assert r(opt=fm.seqs_opts(window=-1)) == fm.FM_ERR_ARG
    assert r(opt=fm.fm_seqs_opts(0.0, 2, 0)) == fm.FM_ERR_ARG
    assert r(opt=fm.seqs_opts(softmax_scale=float("inf"))) == fm.FM_ERR_ARG
    assert r(seqs=fm.fm_seqs(-1, FAKE, FAKE, FAKE, FAKE, 10, 10)) == fm.FM_ERR_ARG
    assert r(seqs=fm.fm_seqs(fm.FM_MAX_SEQS + 1, FAKE, FAKE, FAKE, FAKE, 10, 10)) == fm.FM_ERR_UNSUPPORTED
    assert r(seqs=fm.fm_seqs(3, None, FAKE, FAKE, FAKE, 10, 10)) == fm.FM_ERR_ARG
    assert r(seqs=fm.fm_seqs(3, FAKE, None, None, FAKE, 10, 10)) == fm.FM_ERR_ARG
    assert r(nbytes=1000) == fm.FM_ERR_ARG and "workspace" in fm.fm_last_error()
    assert r(ws=None) == fm.FM_ERR_ARG
    assert r(ws=FAKE + 4) == fm.FM_ERR_ARG
    assert r(lse=FAKE + 2) == fm.FM_ERR_ARG
    assert r(seqs=fm.fm_seqs(0, None, None, None, None, 0, 0)) == fm.FM_OK   # no request: nothing to do
    if paged:
        assert r(seqs=fm.fm_seqs(3, FAKE, FAKE, FAKE, FAKE, 9, 10)) == fm.FM_ERR_ARG  # overlapping table rows
        assert r(seqs=fm.fm_seqs(3, FAKE, FAKE, FAKE, None, 10, 10)) == fm.FM_ERR_ARG
        assert r(k=view(40, 2, 0, 128)) == fm.FM_ERR_SHAPE
    else:
        assert r(k=view(2, 2, 300, 128)) == fm.FM_ERR_SHAPE


def test_workspace_size(lib):
    one = fm.fm_attn_seqs_workspace_size(1, 1, 8, 8, 128)
    assert one > 0
    assert fm.fm_attn_seqs_workspace_size(64, 1000, 8, 8, 128) >= fm.fm_attn_seqs_workspace_size(64, 64, 8, 8, 128) >= one
    for bad in ((-1, 1, 8, 8, 128), (1, -1, 8, 8, 128), (fm.FM_MAX_SEQS + 1, 1, 8, 8, 128), (1, 1, 7, 2, 128),
                (1, 1, 130, 2, 128), (1, 1, 0, 0, 128)):
        with pytest.raises(fm.FMError):
            fm.fm_attn_seqs_workspace_size(*bad)


def test_workspace_size_never_shrinks(lib):
    """Also where a larger call goes to another kernel or another tile of rows."""
    for Hq, Hk in ((1, 1), (5, 1), (10, 2), (16, 1), (64, 1)):
        sizes = [[fm.fm_attn_seqs_workspace_size(n, T, Hq, Hk, 64) for T in (1, 2, 7, 8, 9, 33, 500, 9000)]
                 for n in (1, 2, 3, 30, 31, 500, 8192)]
        for row in sizes:
            assert row == sorted(row)
        for column in zip(*sizes):
            assert list(column) == sorted(column)


def state(**kw):
    d = dict(n_seqs=4, page_size=16, num_pages=32, block_table=FAKE, table_stride=8, table_width=8, free_pages=FAKE,
             free_count=FAKE, free_count_out=FAKE, kv_len=FAKE, kv_len_out=FAKE)
    d.update(kw)
    return fm.fm_page_state(**d)


def extend(lib, st, new_len=FAKE, cap=10, cu=FAKE, slots=FAKE, pos=FAKE, status=FAKE):
    return lib.fm_paged_extend(ctypes.byref(st), new_len, None, cap, cu, slots, pos, status, None)


def test_extend_refusals(lib):
    assert lib.fm_paged_extend(None, FAKE, None, 1, FAKE, FAKE, FAKE, FAKE, None) == fm.FM_ERR_ARG
    for kw in (dict(n_seqs=-1), dict(page_size=0), dict(num_pages=-1), dict(table_width=-1), dict(table_stride=7),
               dict(free_pages=None), dict(free_count=None), dict(free_count_out=None), dict(kv_len=None),
               dict(kv_len_out=None), dict(block_table=None), dict(kv_len=FAKE + 2)):
        assert extend(lib, state(**kw)) == fm.FM_ERR_ARG, kw
    assert extend(lib, state(n_seqs=fm.FM_MAX_SEQS + 1)) == fm.FM_ERR_UNSUPPORTED
    for kw in (dict(new_len=None), dict(cap=-1), dict(cu=None), dict(slots=None), dict(pos=None), dict(status=None),
               dict(slots=FAKE + 4)):
        assert extend(lib, state(), **kw) == fm.FM_ERR_ARG, kw


def test_write_refusals(lib):
    def write(k=None, v=None, kc=None, vc=None, slots=FAKE):
        k, kc = k or view(1, 2, 50, 128), kc or view(9, 2, 16, 128)
        return lib.fm_paged_write(ctypes.byref(k), ctypes.byref(v or k), slots, ctypes.byref(kc), ctypes.byref(vc or kc), None)
    assert write(k=view(2, 2, 50, 128)) == fm.FM_ERR_SHAPE
    assert write(v=view(1, 2, 51, 128)) == fm.FM_ERR_SHAPE
    assert write(kc=view(9, 3, 16, 128)) == fm.FM_ERR_SHAPE
    assert write(vc=view(9, 2, 32, 128)) == fm.FM_ERR_SHAPE
    assert write(kc=view(9, 2, 16, 128, fm.FM_F16)) == fm.FM_ERR_DTYPE
    assert write(slots=None) == fm.FM_ERR_ARG
    assert write(k=view(1, 2, 0, 128)) == fm.FM_OK  # no row: nothing to do


def test_struct_layouts_match_header(tmp_path):
    structs = {"fm_seqs_opts": fm.fm_seqs_opts, "fm_seqs": fm.fm_seqs, "fm_page_state": fm.fm_page_state}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "fm.h"', "int main(void) {"]
    for name, cls in structs.items():
        lines.append(f'  printf("{name} size %zu\\n", sizeof({name}));')
        lines += [f'  printf("{name} {f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["  return 0;", "}"]) + "\n")
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    seen = 0
    for ln in subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.splitlines():
        name, field, val = ln.split()
        got = ctypes.sizeof(structs[name]) if field == "size" else getattr(structs[name], field).offset
        assert got == int(val), (name, field)
        seen += 1
    assert seen == sum(len(c._fields_) + 1 for c in structs.values())


def test_packed_arguments_match_the_structs():
    """What the binding packs is what the ctypes mirrors hold, field by field."""
    t = torch.empty(7, 3, 2, 64, dtype=torch.float16).transpose(1, 2)
    got, want = fm.fm_tensor.from_buffer_copy(fm._cache(t, "t", -1)), fm.tensor(t)
    for f in ("ptr", "dtype", "reserved", "B", "H", "S", "D"):
        assert getattr(got, f) == getattr(want, f), f
    assert list(got.stride) == list(want.stride)
    r = torch.empty(9, 5, 128)[:, 1:3]
    got, want = fm.fm_tensor.from_buffer_copy(fm._rows(r, "r", -1)), fm.tensor(r.permute(1, 0, 2)[None])
    assert [got.ptr, got.dtype, got.B, got.H, got.S, got.D] == [want.ptr, want.dtype, 1, 2, 9, 128]
    assert list(got.stride)[1:] == list(want.stride)[1:]
    s = fm.fm_seqs.from_buffer_copy(fm._SEQS_BYTES(*range(1, 8)))
    assert [getattr(s, f) for f, _ in s._fields_] == list(range(1, 8))
    p = fm.fm_page_state.from_buffer_copy(fm._STATE_BYTES(*range(1, 12)))
    assert [getattr(p, f) for f, _ in p._fields_] == list(range(1, 12))
    assert len(fm._STATE_BYTES(*range(11))) == ctypes.sizeof(fm.fm_page_state)


def test_constants_match_header():
    text = open(os.path.join(ROOT, "include", "fm.h")).read()
    for name in ("FM_MAX_GROUP", "FM_MAX_SEQS"):
        assert f"#define {name} {getattr(fm, name)}\n" in text


def test_binding_refuses_host_tensors(lib, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    cache = torch.zeros(3, 2, 16, 128, dtype=torch.bfloat16)
    slots = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(fm.FMError, match="CUDA device"):
        fm.fm_attn_varlen(q, q, q, i(2), i(2), fm.seqs_opts(), q)
    with pytest.raises(fm.FMError, match="CUDA device"):
        fm.fm_attn_paged(q, cache, cache, i(2), i(1), i(1, 4), fm.seqs_opts(), q)
    with pytest.raises(fm.FMError, match="CUDA device"):
        fm.fm_paged_write(q, q, slots, cache, cache)
    with pytest.raises(fm.FMError, match="CUDA device"):
        fm.fm_paged_extend(i(2), None, i(2), i(2), i(2, 4), i(8), i(1), i(1), 16, i(3), slots, i(4), i(1))


def test_binding_checks_integer_tensors():
    with pytest.raises(fm.FMError, match="cu_q"):
        fm._ints(torch.zeros(3, dtype=torch.int64), torch.int32, 1, "cu_q", 0)
    with pytest.raises(fm.FMError, match="kv_len"):
        fm._ints(torch.zeros(3, dtype=torch.int32), torch.int32, 4, "kv_len", 0)
    with pytest.raises(fm.FMError, match="slots"):
        fm._ints(torch.zeros(6, dtype=torch.int64)[::2], torch.int64, 3, "slots", 0)
    with pytest.raises(fm.FMError, match="block_table"):
        fm._table(torch.zeros(3, 4, dtype=torch.int32).t(), 3, 0)
    with pytest.raises(fm.FMError, match="block_table"):
        fm._table(torch.zeros(2, 4, dtype=torch.int32), 3, 0)


@pytest.mark.parametrize("ws", [torch.empty(1, dtype=torch.uint8).expand(1 << 30), torch.empty(1 << 16, dtype=torch.uint8)[::2],
                                torch.empty(64, 128).t()], ids=["expanded", "every other byte", "transposed"])
@pytest.mark.parametrize("paged", [False, True])
def test_binding_refuses_a_workspace_that_is_no_range_of_bytes(lib, monkeypatch, ws, paged):
    """One byte expanded to a gigabyte passes for a workspace by its number of elements."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # (where get_device() says that host tensors are)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q, cache = torch.zeros(4, 2, 128), torch.zeros(3, 2, 16, 128)
    with pytest.raises(fm.FMError, match="contiguous") as e:
        if paged:
            fm.fm_attn_paged(q, cache, cache, i(2), i(1), i(1, 4), fm.seqs_opts(), q, None, ws, stream=0)
        else:
            fm.fm_attn_varlen(q, q, q, i(2), i(2), fm.seqs_opts(), q, None, ws, stream=0)
    assert e.value.code == fm.FM_ERR_ARG


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("scale", [float("nan"), float("inf"), 3.0e38, 2.4e38])
def test_a_softmax_scale_that_is_no_number_is_refused(lib, paged, scale):
    """NaN does not select the default, and a scale that overflows when taken to base 2 (2.36e38 and more) is as
    infinite as infinity."""
    assert attn(lib, paged, opt=fm.seqs_opts(softmax_scale=scale)) == fm.FM_ERR_ARG
    assert "softmax_scale" in fm.fm_last_error()


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("scale", [0.0, -1.0, float("-inf"), 1e-45, 1e38])
def test_a_softmax_scale_that_is_one_gets_past_that_check(lib, paged, scale):
    assert attn(lib, paged, opt=fm.seqs_opts(softmax_scale=scale), nbytes=1000) == fm.FM_ERR_ARG
    assert "workspace" in fm.fm_last_error()


@pytest.mark.parametrize("window,held", [(0, 0), (7, 7), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1), (2 ** 32, 2 ** 31 - 1),
                                         (2 ** 32 + 5, 2 ** 31 - 1), (2 ** 63 - 1, 2 ** 31 - 1), (-1, -1), (-2 ** 32, -1)])
def test_a_window_past_32_bits_is_not_cut_to_its_low_bits(window, held):
    """2^32 + 5 is no window of 5 keys, -2^32 not none."""
    assert fm.seqs_opts(window=window).window == held


def test_layers_that_share_tables_share_their_limits():
    """A second layer asked for more rows, wider tables or more tokens does not get the first one's without a word."""
    make = lambda *limits, device="cpu", **kw: fm.PagedKVCache(6, 4, 2, 64, *limits, device=device, **kw)  # noqa: E731
    first = make(3, 5, 7)
    second = fm.PagedKVCache(6, 4, 1, 128, 3, 5, 7, dtype=torch.float32, device="cpu", shared=first)
    assert second.kv_len is first.kv_len and second.slots is first.slots and second.k.shape == (6, 1, 4, 128)
    for limits in ((4, 5, 7), (3, 6, 7), (3, 5, 8), (2, 5, 7)):
        with pytest.raises(fm.FMError, match="max_seqs") as e:
            make(*limits, shared=first)
        assert e.value.code == fm.FM_ERR_SHAPE
    with pytest.raises(fm.FMError, match="one device"):
        make(3, 5, 7, device="meta", shared=first)
    with pytest.raises(fm.FMError, match="same pages"):
        fm.PagedKVCache(6, 8, 2, 64, 3, 5, 7, device="cpu", shared=first)
