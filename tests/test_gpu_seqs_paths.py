"""The variants of the serving attention that only some sizes and layouts reach, each against the plain 64-bit
computation: long packed prompts at D = 64, pages whose pitch no grouped tensor map describes, windows at D = 64 and
in fp16, work lists of more than one pass of the planning CTA with cut units among them, batches of mostly idle rows;
the largest number of requests, and calls of nothing."""
import pytest
import torch

import fixed_max_softmax_gb300 as fm
from tests.seqs_reference import assert_close, attend
from tests.test_gpu_seqs import (BF16, DECODE, F16, F32, MIXED, check_paged, check_varlen, dev, paged_case, rand,  # noqa: F401
                                 run_paged, run_varlen, starts)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lens,causal,window", [([(4100, 4100)], True, 0), ([(4095, 4095)], True, 0), ([(4096, 4333)], False, 0),
                                                ([(5000, 5000), (3300, 3300)], True, 0), ([(4200, 4200), (4001, 90)], True, 0),
                                                ([(4500, 4500)], True, 300), ([(4100, 4600), (4200, 4200)], True, 1)])
def test_long_packed_prompts_of_64_columns(dev, dtype, lens, causal, window):  # noqa: F811
    """A mean of 4,096 queries and more (and one below it) at D = 64: whole and cut units, row tiles alone and in pairs,
    more queries than keys, rows that see one key."""
    g = torch.Generator(device=dev).manual_seed(50)
    T, Tk = sum(a for a, _ in lens), sum(b for _, b in lens)
    q, k, v = (rand(g, n, h, 64, dtype=dtype, scale=s) for n, h, s in ((T, 2, 1.5), (Tk, 1, 1.0), (Tk, 1, 1.0)))
    o, lse = run_varlen(q, k, v, lens, causal, window, dev=dev)
    check_varlen(q, k, v, lens, o, lse, causal, window)


def test_long_packed_prompts_uncut(dev):  # noqa: F811
    """So many units that none is cut: 3 prompts, 16 key heads of 4 query heads; the first and last key heads of one."""
    g = torch.Generator(device=dev).manual_seed(51)
    lens, Hk, G = [(4100, 4100), (4200, 4200), (4000, 4000)], 16, 4
    T = sum(a for a, _ in lens)
    q, k, v = rand(g, T, Hk * G, 64, dtype=BF16), rand(g, T, Hk, 64, dtype=BF16), rand(g, T, Hk, 64, dtype=BF16)
    o, lse = run_varlen(q, k, v, lens, dev=dev)
    at = slice(4100, 8300)
    for h in (0, Hk - 1):
        hs = slice(h * G, h * G + G)
        r = attend(q[at, hs], k[at, h:h + 1], v[at, h:h + 1], True, 0, 0.125)
        assert_close(o[at, hs], lse[hs, at], *r, BF16, BF16, 64, 4200)


def pitched(cache, token_major, pad):
    """The same cache with `pad` elements of NaN between its pages."""
    pages, Hk, ps, D = cache.shape
    flat = torch.full((pages, Hk * ps * D + pad), float("nan"), dtype=cache.dtype, device=cache.device)
    body = flat[:, :Hk * ps * D]
    out = body.view(pages, ps, Hk, D).transpose(1, 2) if token_major else body.view(pages, Hk, ps, D)
    out.copy_(cache)
    assert out.stride(0) == Hk * ps * D + pad
    return out


@pytest.mark.parametrize("token_major", [True, False])
@pytest.mark.parametrize("ps", [8, 16, 32, 64, 128])
@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F16, 64)])
@pytest.mark.parametrize("pads", ["no group", "keys alone", "whole groups", "unaligned"])
@pytest.mark.parametrize("lens", [DECODE, MIXED])
def test_page_pitch(dev, token_major, ps, dtype, D, pads, lens):  # noqa: F811
    """Pages that lie no whole number of 8-row groups apart, keys and values of different pitches, a pitch of whole
    groups larger than the page, and one that is no multiple of 16 bytes."""
    g = torch.Generator(device=dev).manual_seed(52)
    Hk = 2
    ks, vs, kc, vc, table = paged_case(g, lens, Hk, D, ps, dtype, token_major)
    group = 8 * (Hk * D if token_major else D)  # elements of 8 rows
    k_pad, v_pad = {"no group": (64, 64), "keys alone": (group, 0), "whole groups": (group, group), "unaligned": (4, 4)}[pads]
    q = rand(g, sum(a for a, _ in lens), 10, D, dtype=dtype)
    o, lse = run_paged(q, pitched(kc, token_major, k_pad), pitched(vc, token_major, v_pad), table, lens, dev)
    fm.fm_sync_status()
    check_paged(q, ks, vs, lens, o, lse)


@pytest.mark.parametrize("dtype,D", [(BF16, 64), (F16, 64), (F16, 128)])
@pytest.mark.parametrize("ps", [8, 32, 64, 128, 256])
@pytest.mark.parametrize("window,lens", [(50, [(1, 700), (1, 30), (1, 300)]), (130, [(60, 900), (1, 1), (5, 640)]),
                                         (700, [(300, 2000), (1, 1500), (90, 130)])])
def test_keys_before_the_window_at_64_columns_and_in_fp16(dev, dtype, D, ps, window, lens):  # noqa: F811
    """Rows before every query's window hold NaN, and whole such pages' table entries point outside the cache."""
    g = torch.Generator(device=dev).manual_seed(53)
    ks, vs, kc, vc, table = paged_case(g, lens, 2, D, ps, dtype, True)
    for i, (a, b) in enumerate(lens):
        first = max(0, b - a - window + 1)  # the oldest key that the first query sees
        for j in range(first // ps + 1):
            rows = min(ps, first - j * ps)
            if rows > 0:
                kc[table[i, j], :, :rows] = float("nan")
                vc[table[i, j], :, :rows] = float("nan")
            if rows == ps:
                table[i, j] = -1
    q = rand(g, sum(a for a, _ in lens), 8, D, dtype=dtype)
    o, lse = run_paged(q, kc, vc, table, lens, dev, window=window)
    fm.fm_sync_status()
    check_paged(q, ks, vs, lens, o, lse, window=window)


@pytest.mark.parametrize("dtype,D", [(BF16, 64), (F16, 64), (F16, 128), (F32, 64)])
@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 17), (True, 128), (True, 700)])
def test_masks_at_64_columns_and_in_fp16(dev, dtype, D, causal, window):  # noqa: F811
    g = torch.Generator(device=dev).manual_seed(54)
    lens = [(260, 260), (1, 900), (50, 1400), (30, 8), (600, 600)]
    T, Tk = sum(a for a, _ in lens), sum(b for _, b in lens)
    q, k, v = (rand(g, n, h, D, dtype=dtype) for n, h in ((T, 8), (Tk, 2), (Tk, 2)))
    o, lse = run_varlen(q, k, v, lens, causal, window, dev=dev)
    check_varlen(q, k, v, lens, o, lse, causal, window)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_long_work_list_with_cut_units(dev, dtype):  # noqa: F811
    """1,200 (fp32: 4,800) pieces of one prompt, which no unit of it is cut into, between two requests whose units
    are: the planning CTA writes such a list in several passes.  Key heads 0, 9 and 15 of 16."""
    g = torch.Generator(device=dev).manual_seed(55)
    lens, Hk, G, D = [(4, 20000), (1200, 1200), (4, 20000)], 16, 16, 64
    ks, vs, kc, vc, table = paged_case(g, lens, Hk, D, 16, dtype, True)
    q = rand(g, sum(a for a, _ in lens), Hk * G, D, dtype=dtype)
    o, lse = run_paged(q, kc, vc, table, lens, dev)
    fm.fm_sync_status()
    for h in (0, 9, 15):
        hs = slice(h * G, h * G + G)
        check_paged(q[:, hs], [k[:, h:h + 1] for k in ks], [v[:, h:h + 1] for v in vs], lens, o[:, hs], lse[hs])


@pytest.mark.parametrize("dtype,tokens", [(BF16, 3000), (F32, 500), (F32, 1400)])
def test_one_prompt_in_a_batch_of_idle_rows(dev, dtype, tokens):  # noqa: F811
    """256 rows of which three hold requests: the prompt goes the way of a decoding batch."""
    g = torch.Generator(device=dev).manual_seed(56)
    lens = [(0, 0)] * 256
    lens[7], lens[100], lens[255] = (1, 300), (tokens, tokens), (3, 50)
    ks, vs, kc, vc, table = paged_case(g, lens, 1, 64, 16, dtype, True)
    q = rand(g, tokens + 4, 4, 64, dtype=dtype)
    o, lse = run_paged(q, kc, vc, table, lens, dev)
    fm.fm_sync_status()
    check_paged(q, ks, vs, lens, o, lse)


@pytest.mark.parametrize("dtype,D", [(BF16, 64), (BF16, 128), (F32, 64)])
def test_decoding_rows_in_long_buffers(dev, dtype, D):  # noqa: F811
    """24 single tokens in buffers of 2,048 rows, as a captured step has them: rows behind the last are left alone."""
    g = torch.Generator(device=dev).manual_seed(57)
    lens = [(1, 40 + 97 * i) for i in range(24)]
    ks, vs, kc, vc, table = paged_case(g, lens, 2, D, 16, dtype, True)
    q = rand(g, 2048, 10, D, dtype=dtype)
    q[24:] = float("nan")
    o, lse = run_paged(q, kc, vc, table, lens, dev)
    fm.fm_sync_status()
    check_paged(q[:24], ks, vs, lens, o[:24], lse[:, :24])
    assert (o[24:] == 7.0).all() and (lse[:, 24:] == 7.0).all()
    assert starts([a for a, _ in lens])[-1] == 24


@pytest.mark.parametrize("dtype,G,tokens", [(BF16, 4, 1), (F16, 16, 9), (F32, 4, 1), (F32, 16, 1), (F32, 16, 5)])
def test_the_largest_number_of_requests(dev, dtype, G, tokens):  # noqa: F811
    """FM_MAX_SEQS requests: even runs and a work list on the tensor cores, units of 8, 16 and 64 rows on the CUDA cores;
    a sample of the requests, those in the last pass of the planning CTA among them."""
    g = torch.Generator(device=dev).manual_seed(58)
    n, D = fm.FM_MAX_SEQS, 64
    lens = [(tokens, tokens + (i * 7) % 40) for i in range(n)]
    lens[5000] = (tokens, 3000)
    cq, ck = starts([a for a, _ in lens]), starts([b for _, b in lens])
    q, k, v = (rand(g, t, h, D, dtype=dtype) for t, h in ((cq[-1], G), (ck[-1], 1), (ck[-1], 1)))
    o, lse = run_varlen(q, k, v, lens, dev=dev)
    for i in (0, 1, 383, 384, 1023, 1024, 4999, 5000, 5001, 7167, 7168, n - 2, n - 1):
        a, b = slice(cq[i], cq[i + 1]), slice(ck[i], ck[i + 1])
        r = attend(q[a], k[b], v[b], True, 0, D ** -0.5)
        assert_close(o[a], lse[:, a], *r, dtype, dtype, D, lens[i][1])
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("n,cap", [(8192, 9000), (8192, 3000)])
def test_extend_of_the_largest_number_of_requests(dev, n, cap):  # noqa: F811
    """One token each in place (as many as the slots hold), by one CTA and by the two kernels."""
    t32 = dict(dtype=torch.int32, device=dev)
    new = torch.zeros(n, **t32)
    new[:min(n, cap)] = 1
    kv = (torch.arange(n, device=dev) % 4).int()  # pages of 4: none, or one that the token still fits
    held = int((kv > 0).sum())
    pages = n + 3
    table = torch.full((n, 2), -1, **t32)
    table[kv > 0, 0] = torch.arange(held, **t32)
    free = torch.full((pages,), -1, **t32)
    free[:pages - held] = torch.arange(held, pages, **t32)
    count, cu, status = torch.tensor([pages - held], **t32), torch.zeros(n + 1, **t32), torch.full((1,), 9, **t32)
    slots, pos = torch.full((cap,), 9, dtype=torch.int64, device=dev), torch.full((cap,), 9, **t32)
    fresh = ((kv == 0) & (new == 1)).cpu()
    page = table[:, 0].cpu().long()
    page[fresh] = free.cpu().long()[pages - held - 1 - torch.arange(int(fresh.sum()))]
    want = (page * 4 + kv.cpu().long())[:min(n, cap)]
    want_pos, want_kv = kv.cpu()[:min(n, cap)], kv + new
    fm.fm_paged_extend(new, None, kv, kv, table, free, count, count, 4, cu, slots, pos, status)
    fm.fm_sync_status()
    assert status.item() == 0 and torch.equal(kv, want_kv) and count.item() == pages - held - int(fresh.sum())
    assert torch.equal(slots[:len(want)].cpu(), want) and torch.equal(pos[:len(want)].cpu(), want_pos)
    assert (slots[len(want):] == -1).all() and (pos[len(want):] == -1).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_no_pages_no_keys_no_queries(dev, dtype):  # noqa: F811
    """Caches of no page, tables of no column, keys of no row: every query sees nothing.  And calls of no query."""
    q = torch.ones(5, 4, 64, dtype=dtype, device=dev)
    none = torch.empty(0, 2, 16, 64, dtype=dtype, device=dev)
    lens = [(2, 0), (0, 0), (3, 0)]
    for pages in (none, torch.full((3, 2, 16, 64), float("nan"), dtype=dtype, device=dev)):
        o, lse = run_paged(q, pages, pages, torch.empty(3, 0, dtype=torch.int32, device=dev), lens, dev)
        fm.fm_sync_status()
        assert (o == 0).all() and torch.isneginf(lse).all()
    rows = torch.empty(0, 2, 64, dtype=dtype, device=dev)
    o, lse = run_varlen(q, rows, rows, lens, dev=dev)
    assert (o == 0).all() and torch.isneginf(lse).all()
    o, lse = run_varlen(q[:0], rows, rows, [(0, 0)] * 3, dev=dev)
    assert o.numel() == lse.numel() == 0
    c = fm.PagedKVCache(3, 16, 2, 64, 2, 1, 4, dtype=dtype, device=dev)
    c.extend(torch.zeros(2, dtype=torch.int32, device=dev))
    c.write(rows, rows)
    assert c.attention(q[:0]).shape == (0, 4, 64)
    assert not c.attention(q).any()  # five rows behind the last token
    fm.fm_sync_status()
    assert c.status.tolist() == [0]
