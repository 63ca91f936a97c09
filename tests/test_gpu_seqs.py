"""Attention over requests of different lengths and the paged cache, on the GPU, against a plain
64-bit computation (tests/seqs_reference.py, whose bounds count the roundings)."""
import math
import random

import pytest
import torch

import fixed_max_softmax_gb300 as fm
from tests.seqs_reference import assert_close, attend

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def dev():
    from fixed_max_softmax_gb300 import build as fmbuild

    fmbuild.build()
    fm.load()
    torch.cuda.set_device(0)
    return torch.device("cuda:0")


def ints(v, dev, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=dev)


def starts(lens):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return cu


def rand(g, *shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device=g.device) * scale).to(dtype)


def workspace(n, T, Hq, Hk, D, dev):
    ws = torch.empty(fm.fm_attn_seqs_workspace_size(n, T, Hq, Hk, D), dtype=torch.uint8, device=dev)
    ws.fill_(0xFF)  # its contents need no preparation: NaN patterns and negative counts
    return ws


def run_varlen(q, k, v, lens, causal=True, window=0, scale=0.0, out_dtype=None, dev=None):
    ql, kl = [a for a, _ in lens], [b for _, b in lens]
    T, Hq, D = q.shape
    o = torch.full((T, Hq, D), 7.0, dtype=out_dtype or q.dtype, device=dev)
    lse = torch.full((Hq, T), 7.0, device=dev)
    fm.fm_attn_varlen(q, k, v, ints(starts(ql), dev), ints(starts(kl), dev), fm.seqs_opts(causal, window, scale), o, lse,
                      workspace(len(lens), T, Hq, k.shape[1], D, dev))
    fm.fm_sync_status()
    return o, lse


def check_varlen(q, k, v, lens, o, lse, causal, window, scale=0.0):
    D = q.shape[2]
    cq, ck = starts([a for a, _ in lens]), starts([b for _, b in lens])
    for i, (a, b) in enumerate(lens):
        r = attend(q[cq[i]:cq[i + 1]], k[ck[i]:ck[i + 1]], v[ck[i]:ck[i + 1]], causal, window, scale or D ** -0.5)
        assert_close(o[cq[i]:cq[i + 1]], lse[:, cq[i]:cq[i + 1]], *r, q.dtype, o.dtype, D, b)


LENGTHS = {
    "one token": [(1, 1)],
    "prompts": [(5, 5), (1, 1), (130, 130), (0, 0), (257, 257)],
    "chunks": [(3, 90), (64, 200), (1, 515), (40, 41)],
    "no keys": [(2, 0), (3, 3), (0, 5), (1, 0)],
    "more queries than keys": [(20, 7), (200, 130)],
    "one long": [(7, 3001)],
    "longer": [(300, 1500), (1, 2300)],
}


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F16, 128), (BF16, 64), (F16, 64), (F32, 128), (F32, 64)])
@pytest.mark.parametrize("name", list(LENGTHS))
def test_varlen_lengths(dev, name, dtype, D):
    g = torch.Generator(device=dev).manual_seed(1)
    lens = LENGTHS[name]
    Hq, Hk = 6, 2
    T, Tk = sum(a for a, _ in lens), sum(b for _, b in lens)
    q = rand(g, T, Hq, D, dtype=dtype, scale=1.5)
    k, v = rand(g, Tk, Hk, D, dtype=dtype), rand(g, Tk, Hk, D, dtype=dtype)
    o, lse = run_varlen(q, k, v, lens, dev=dev)
    check_varlen(q, k, v, lens, o, lse, True, 0)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (5, 1), (7, 7), (14, 2), (24, 3), (32, 1), (64, 1), (33, 3)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_varlen_heads(dev, Hq, Hk, dtype):
    g = torch.Generator(device=dev).manual_seed(2)
    lens = [(70, 70), (1, 300), (9, 140)]
    T, Tk = 80, 510
    q = rand(g, T, Hq, 128, dtype=dtype)
    k, v = rand(g, Tk, Hk, 128, dtype=dtype), rand(g, Tk, Hk, 128, dtype=dtype)
    o, lse = run_varlen(q, k, v, lens, dev=dev)
    check_varlen(q, k, v, lens, o, lse, True, 0)


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 2), (True, 17), (True, 128), (True, 130),
                                           (True, 700), (True, 100000), (True, 2 ** 31 - 1)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_varlen_masks(dev, causal, window, dtype):
    g = torch.Generator(device=dev).manual_seed(3)
    lens = [(260, 260), (1, 900), (50, 1400), (30, 8), (600, 600)]
    T, Tk = sum(a for a, _ in lens), sum(b for _, b in lens)
    q, k, v = (rand(g, n, h, 128, dtype=dtype) for n, h in ((T, 8), (Tk, 2), (Tk, 2)))
    o, lse = run_varlen(q, k, v, lens, causal, window, dev=dev)
    check_varlen(q, k, v, lens, o, lse, causal, window)


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
def test_sharp_rows_and_scale(dev, dtype):
    """Scores far apart (one key takes nearly all the weight), growing along the keys, so that the
    running max moves again and again; and another softmax scale."""
    g = torch.Generator(device=dev).manual_seed(4)
    lens = [(150, 700)]
    q, k, v = (rand(g, n, h, 128, dtype=dtype) for n, h in ((150, 4), (700, 2), (700, 2)))
    k = (k.float() * torch.linspace(0.1, 6.0, 700, device=dev)[:, None, None]).to(dtype)
    o, lse = run_varlen(q, k, v, lens, scale=0.2, dev=dev)
    check_varlen(q, k, v, lens, o, lse, True, 0, 0.2)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strides_fp32_output_and_rows_behind_the_last(dev, dtype):
    """q, k, v as slices of one fused buffer, o inside a wider one, [1, H, T, D] views; rows behind
    the last request are neither read (they hold NaN) nor written."""
    g = torch.Generator(device=dev).manual_seed(5)
    lens = [(60, 60), (33, 33)]
    T, extra, Hq, Hk, D = 93, 11, 8, 2, 128
    fused = rand(g, T + extra, Hq + 2 * Hk, D, dtype=dtype)
    fused[T:] = float("nan")
    q, k, v = fused[:, :Hq], fused[:, Hq:Hq + Hk], fused[:, Hq + Hk:]
    wide = torch.full((T + extra, Hq, D + 32), 3.0, device=dev)
    lse = torch.full((Hq, T + extra), 3.0, device=dev)
    o = wide[..., 16:16 + D]
    cu = ints(starts([a for a, _ in lens]), dev)
    four = lambda t: t.permute(1, 0, 2).unsqueeze(0)  # noqa: E731
    fm.fm_attn_varlen(four(q), four(k), four(v), cu, cu, fm.seqs_opts(), four(o), lse,
                      workspace(2, T + extra, Hq, Hk, D, dev))
    fm.fm_sync_status()
    check_varlen(q[:T], k[:T], v[:T], lens, o[:T], lse[:, :T], True, 0)
    assert (wide[T:] == 3.0).all() and (wide[:, :, :16] == 3.0).all() and (wide[:, :, 16 + D:] == 3.0).all()
    assert (lse[:, T:] == 3.0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_odd_layouts(dev, dtype):
    """Head dimension not adjacent, and rows that are not 16-byte aligned."""
    g = torch.Generator(device=dev).manual_seed(6)
    lens = [(40, 40), (3, 3)]
    q = rand(g, 43, 4, 128, 2, dtype=dtype)[..., 1]
    k, v = rand(g, 43, 2, 131, dtype=dtype)[..., 1:129], rand(g, 43, 2, 128, dtype=dtype)
    o, lse = run_varlen(q, k, v, lens, dev=dev)
    check_varlen(q, k, v, lens, o, lse, True, 0)


def paged_case(g, lens, Hk, D, ps, dtype, token_major, stale=float("nan")):
    """Keys and values of every request, and a cache that holds them on shuffled pages with `stale`
    everywhere else."""
    need = [-(-s // ps) for _, s in lens]
    pages = sum(need) + 5
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(9)).tolist()
    shape = (pages, ps, Hk, D) if token_major else (pages, Hk, ps, D)
    kc, vc = (torch.full(shape, stale, dtype=dtype, device=g.device) for _ in range(2))
    if token_major:
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    table = torch.full((len(lens), max(need + [1]) + 2), 2 ** 31 - 1, dtype=torch.int32)
    ks, vs = [], []
    for i, (_, s) in enumerate(lens):
        k, v = rand(g, s, Hk, D, dtype=dtype), rand(g, s, Hk, D, dtype=dtype)
        for j in range(need[i]):
            p = order.pop()
            table[i, j] = p
            n = min(ps, s - j * ps)
            kc[p, :, :n] = k[j * ps:j * ps + n].transpose(0, 1)
            vc[p, :, :n] = v[j * ps:j * ps + n].transpose(0, 1)
        ks.append(k)
        vs.append(v)
    return ks, vs, kc, vc, table.to(g.device)


def run_paged(q, kc, vc, table, lens, dev, causal=True, window=0):
    T, Hq, D = q.shape
    o, lse = torch.full_like(q, 7.0), torch.full((Hq, T), 7.0, device=dev)
    fm.fm_attn_paged(q, kc, vc, ints(starts([a for a, _ in lens]), dev), ints([b for _, b in lens], dev), table,
                     fm.seqs_opts(causal, window), o, lse, workspace(len(lens), T, Hq, kc.shape[1], D, dev))
    return o, lse


def check_paged(q, ks, vs, lens, o, lse, causal=True, window=0, skip=()):
    cq, D = starts([a for a, _ in lens]), q.shape[2]
    for i, (a, b) in enumerate(lens):
        if i not in skip:
            r = attend(q[cq[i]:cq[i + 1]], ks[i], vs[i], causal, window, D ** -0.5)
            assert_close(o[cq[i]:cq[i + 1]], lse[:, cq[i]:cq[i + 1]], *r, q.dtype, o.dtype, D, b)


DECODE = [(1, 1), (1, 15), (1, 16), (1, 17), (1, 127), (1, 128), (1, 129), (1, 777), (1, 0), (0, 40), (1, 2600)]
MIXED = [(1, 300), (70, 333), (1, 1), (200, 200), (0, 9), (5, 1999)]


@pytest.mark.parametrize("token_major", [True, False])
@pytest.mark.parametrize("ps", [1, 3, 8, 16, 48, 64, 128, 256, 192])
@pytest.mark.parametrize("dtype,lens", [(BF16, DECODE), (BF16, MIXED), (F32, MIXED)])
def test_paged_page_sizes(dev, ps, dtype, lens, token_major):
    g = torch.Generator(device=dev).manual_seed(7)
    ks, vs, kc, vc, table = paged_case(g, lens, 2, 128, ps, dtype, token_major)
    q = rand(g, sum(a for a, _ in lens), 10, 128, dtype=dtype, scale=1.5)
    o, lse = run_paged(q, kc, vc, table, lens, dev)
    fm.fm_sync_status()
    check_paged(q, ks, vs, lens, o, lse)


@pytest.mark.parametrize("dtype,D,Hq,Hk", [(F16, 128, 16, 2), (F16, 64, 7, 7), (BF16, 64, 64, 1), (F32, 64, 8, 8),
                                           (BF16, 128, 1, 1), (BF16, 128, 40, 8)])
@pytest.mark.parametrize("lens", [DECODE, MIXED, [(1, 9000)], [(2, 4000), (1, 30), (128, 6000)]])
def test_paged_types_and_heads(dev, dtype, D, Hq, Hk, lens):
    g = torch.Generator(device=dev).manual_seed(8)
    ks, vs, kc, vc, table = paged_case(g, lens, Hk, D, 16, dtype, True)
    q = rand(g, sum(a for a, _ in lens), Hq, D, dtype=dtype)
    o, lse = run_paged(q, kc, vc, table, lens, dev)
    fm.fm_sync_status()
    check_paged(q, ks, vs, lens, o, lse)


@pytest.mark.parametrize("window", [1, 16, 100, 128, 1000])
@pytest.mark.parametrize("lens", [DECODE, MIXED, [(40, 5000)]])
def test_paged_window(dev, window, lens):
    g = torch.Generator(device=dev).manual_seed(9)
    ks, vs, kc, vc, table = paged_case(g, lens, 2, 128, 16, BF16, True)
    q = rand(g, sum(a for a, _ in lens), 8, 128, dtype=BF16)
    o, lse = run_paged(q, kc, vc, table, lens, dev, window=window)
    fm.fm_sync_status()
    check_paged(q, ks, vs, lens, o, lse, window=window)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("ps", [8, 16, 64, 128])
@pytest.mark.parametrize("window,lens", [(50, [(1, 700), (1, 30), (1, 300)]), (130, [(60, 900), (1, 1), (5, 640)])])
def test_keys_before_the_window_may_hold_anything(dev, dtype, ps, window, lens):
    """Rows that every query's window has passed hold NaN, and the table entries of whole such pages
    point outside the cache: as after a server has taken those pages back."""
    g = torch.Generator(device=dev).manual_seed(20)
    ks, vs, kc, vc, table = paged_case(g, lens, 2, 128, ps, dtype, True)
    for i, (a, b) in enumerate(lens):
        first = max(0, b - a - window + 1)  # the oldest key that the first query sees
        for j in range(first // ps + 1):
            rows = min(ps, first - j * ps)
            if rows > 0:
                kc[table[i, j], :, :rows] = float("nan")
                vc[table[i, j], :, :rows] = float("nan")
            if rows == ps:
                table[i, j] = -1
    q = rand(g, sum(a for a, _ in lens), 8, 128, dtype=dtype)
    o, lse = run_paged(q, kc, vc, table, lens, dev, window=window)
    fm.fm_sync_status()
    check_paged(q, ks, vs, lens, o, lse, window=window)


def test_offsets_past_32_bits(dev):
    """A cache of more than 2^31 elements, with the request on its last pages: written and read."""
    g = torch.Generator(device=dev).manual_seed(21)
    Hk, D, ps, pages = 8, 128, 16, 135000
    kc, vc = (torch.empty(pages, ps, Hk, D, dtype=BF16, device=dev).transpose(1, 2) for _ in range(2))
    assert kc.numel() > 2 ** 31
    lens = [(1, 200), (3, 100)]
    table = torch.tensor([[pages - 1 - 2 * j for j in range(13)], [pages - 2 - 2 * j for j in range(13)]], dtype=torch.int32)
    ks, vs = ([rand(g, s, Hk, D, dtype=BF16) for _, s in lens] for _ in range(2))
    slots = [int(table[i, p // ps]) * ps + p % ps for i, (_, s) in enumerate(lens) for p in range(s)]
    fm.fm_paged_write(torch.cat(ks), torch.cat(vs), ints(slots, dev, torch.int64), kc, vc)
    q = rand(g, 4, 16, D, dtype=BF16)
    o, lse = run_paged(q, kc, vc, table.to(dev), lens, dev)
    fm.fm_sync_status()
    check_paged(q, ks, vs, lens, o, lse)
    assert torch.equal(kc[table[0, 0], :, 3], ks[0][3])


def test_paged_not_causal_and_shared_pages(dev):
    """Two requests whose tables name the same pages, and every query seeing every key."""
    g = torch.Generator(device=dev).manual_seed(10)
    lens = [(4, 300), (2, 280)]
    ks, vs, kc, vc, table = paged_case(g, [(4, 300)], 2, 128, 16, BF16, True)
    table = table.repeat(2, 1)
    q = rand(g, 6, 8, 128, dtype=BF16)
    o, lse = run_paged(q, kc, vc, table, lens, dev, causal=False)
    fm.fm_sync_status()
    check_paged(q, [ks[0], ks[0][:280]], [vs[0], vs[0][:280]], lens, o, lse, causal=False)


@pytest.mark.parametrize("dtype,ps", [(F32, 16), (F32, 130), (BF16, 24), (F16, 1)])
@pytest.mark.parametrize("Hq,Hk,D,tokens", [(2, 2, 128, 1), (10, 2, 128, 1), (8, 1, 64, 1), (4, 1, 128, 2), (9, 1, 64, 1),
                                            (32, 2, 128, 1), (5, 1, 64, 3)])
@pytest.mark.parametrize("window", [0, 100])
def test_few_rows_on_the_cuda_cores(dev, dtype, ps, Hq, Hk, D, tokens, window):
    """Units of up to 8 and up to 16 rows, whole and cut, rows without a key, and one request of more
    rows than a unit holds."""
    g = torch.Generator(device=dev).manual_seed(41)
    lens = [(tokens, s) for s in (0, tokens, 5, 63, 64, 65, 300, 2100)] + [(0, 70), (tokens + (9 if Hq // Hk < 16 else 0), 400)]
    lens += [(1, 33)] * 12
    assert sum(a for a, _ in lens) * (Hq // Hk) <= 16 * len(lens)
    ks, vs, kc, vc, table = paged_case(g, lens, Hk, D, ps, dtype, True)
    q = rand(g, sum(a for a, _ in lens), Hq, D, dtype=dtype)
    o, lse = run_paged(q, kc, vc, table, lens, dev, window=window)
    fm.fm_sync_status()
    check_paged(q, ks, vs, lens, o, lse, window=window)


def test_a_request_of_millions_of_keys(dev):
    """One request whose table names the same page again and again: the softmax weights of a page,
    its lse plus the log of the repeats.  64 heads x 22,800 tiles, more than any cache here holds."""
    g = torch.Generator(device=dev).manual_seed(40)
    reps, Hk, D, ps = 22800, 64, 64, 128
    k, v = rand(g, ps, Hk, D, dtype=BF16), rand(g, ps, Hk, D, dtype=BF16)
    q = rand(g, 1, Hk, D, dtype=BF16)
    table = torch.zeros(1, reps, dtype=torch.int32, device=dev)
    o, lse = run_paged(q, k.transpose(0, 1)[None], v.transpose(0, 1)[None], table, [(1, reps * ps)], dev)
    fm.fm_sync_status()
    ro, rl, ra, big = attend(q, k, v, True, 0, D ** -0.5)
    # fp32 sums: the weights of a tile are summed first, then the tiles (reps terms); O takes the products
    # of 16 keys at a time, 8 a tile
    assert_close(o, lse, ro, rl + math.log(reps), ra, big, BF16, BF16, D, 8 * reps)


def test_more_tiles_than_a_decoding_call_takes(dev):
    """8,192 requests x 64 heads x 1,025 tiles (a shared page): refused on the device, nothing computed."""
    n, Hk, D, ps = 8192, 64, 64, 128
    kc = torch.zeros(1, Hk, ps, D, dtype=BF16, device=dev)
    q = torch.zeros(n, Hk, D, dtype=BF16, device=dev)
    table = torch.zeros(n, 1025, dtype=torch.int32, device=dev)
    o, lse = run_paged(q, kc, kc, table, [(1, 1025 * ps)] * n, dev)
    with pytest.raises(fm.FMError, match="lengths") as e:
        fm.fm_sync_status()
    assert e.value.code == fm.FM_ERR_INDEX
    assert (o == 7.0).all() and (lse == 7.0).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_requests(dev, dtype):
    g = torch.Generator(device=dev).manual_seed(11)
    r = random.Random(5)
    lens = [(1, r.randint(1, 60)) for _ in range(1500)]
    ks, vs, kc, vc, table = paged_case(g, lens, 1, 64, 16, dtype, True, stale=0.0)
    q = rand(g, 1500, 4, 64, dtype=dtype)
    o, lse = run_paged(q, kc, vc, table, lens, dev)
    fm.fm_sync_status()
    check_paged(q[:100], ks, vs, lens[:100], o[:100], lse[:, :100])
    sel = 1400
    check_paged(q[sel:], ks[sel:], vs[sel:], lens[sel:], o[sel:], lse[:, sel:])


def test_same_bits_twice_and_on_another_stream(dev):
    g = torch.Generator(device=dev).manual_seed(12)
    ks, vs, kc, vc, table = paged_case(g, MIXED, 2, 128, 16, BF16, True)
    q = rand(g, sum(a for a, _ in MIXED), 8, 128, dtype=BF16)
    first = run_paged(q, kc, vc, table, MIXED, dev)
    again = run_paged(q, kc, vc, table, MIXED, dev)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other = run_paged(q, kc, vc, table, MIXED, dev)
    fm.fm_sync_status(s)
    for x in (again, other):
        assert torch.equal(first[0], x[0]) and torch.equal(first[1], x[1])


def test_two_calls_at_once(dev):
    """Two streams with a workspace each."""
    g = torch.Generator(device=dev).manual_seed(13)
    lens = [(1, 3000)] * 6
    a, b = (paged_case(g, lens, 2, 128, 16, BF16, True) for _ in range(2))
    q = [rand(g, 6, 8, 128, dtype=BF16) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [None, None]
    for _ in range(3):
        for i, c in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                outs[i] = run_paged(q[i], c[2], c[3], c[4], lens, dev)
    torch.cuda.synchronize()
    for i, c in enumerate((a, b)):
        check_paged(q[i], c[0], c[1], lens, *outs[i])


def test_captured_and_replayed_with_other_lengths(dev):
    """One graph of the call, replayed after the lengths on the device have changed."""
    g = torch.Generator(device=dev).manual_seed(14)
    lens = [(1, 500), (1, 1300), (1, 40)]
    ks, vs, kc, vc, table = paged_case(g, lens, 2, 128, 16, BF16, True)
    q = rand(g, 3, 8, 128, dtype=BF16)
    o, lse = torch.empty_like(q), torch.empty(8, 3, device=dev)
    cu, kv, ws = ints([0, 1, 2, 3], dev), ints([5, 5, 5], dev), workspace(3, 3, 8, 2, 128, dev)
    opt = fm.seqs_opts()
    fm.fm_attn_paged(q, kc, vc, cu, kv, table, opt, o, lse, ws)  # the first call comes before a capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fm.fm_attn_paged(q, kc, vc, cu, kv, table, opt, o, lse, ws)
    for now in ([500, 1300, 40], [1, 7, 0], [300, 1024, 33]):
        kv.copy_(ints(now, dev))
        graph.replay()
        fm.fm_sync_status()
        check_paged(q, [k[:n] for k, n in zip(ks, now)], [v[:n] for v, n in zip(vs, now)], [(1, n) for n in now], o, lse)


def test_a_captured_call_may_be_the_first_of_its_kind(tmp_path):
    """After one call on the device, calls that take other kernels (types, page sizes, prompts instead
    of single tokens) can be captured though none of them has run: in a process of its own."""
    import subprocess
    import sys

    code = """
import torch, fixed_max_softmax_gb300 as fm
dev = torch.device("cuda:0")
def call(dtype, T, n, D, ps, out):
    q = torch.ones(T, 4, D, dtype=dtype, device=dev)
    kc = torch.ones(200 // ps + 2, 2, ps, D, dtype=dtype, device=dev)
    cu = torch.tensor([0] + [T // n * (i + 1) for i in range(n)], dtype=torch.int32, device=dev)
    kv = torch.full((n,), 190, dtype=torch.int32, device=dev)
    table = torch.arange(200 // ps + 1, dtype=torch.int32, device=dev).repeat(n, 1)
    ws = torch.empty(fm.fm_attn_seqs_workspace_size(n, T, 4, 2, D), dtype=torch.uint8, device=dev)
    o = torch.zeros_like(q)
    out.append((q, kc, cu, kv, table, ws, o))
    return lambda: fm.fm_attn_paged(q, kc, kc, cu, kv, table, fm.seqs_opts(), o, None, ws)
bufs = []
call(torch.float32, 2, 2, 64, 16, bufs)()
todo = [call(d, T, n, D, ps, bufs) for d in (torch.bfloat16, torch.float16, torch.float32) for D in (64, 128)
        for T, n in ((2, 2), (160, 1)) for ps in (16, 128, 5)]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    for f in todo:
        f()
for b in bufs[1:]:
    assert not b[-1].any()
g.replay()
fm.fm_sync_status()
for b in bufs:  # equal weights and values of one: two sums of at most 190 equal fp32 terms, in different orders
    assert ((b[-1].float() - 1).abs() <= 2 * 198 * 2.0 ** -24).all(), b[0].dtype
print("fine")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("entry", [-1, 1000, 2 ** 31 - 1, -2 ** 31])
def test_bad_page_reads_zeros_and_is_reported(dev, dtype, entry):
    g = torch.Generator(device=dev).manual_seed(15)
    lens = [(1, 100), (2, 200), (1, 64)]
    ks, vs, kc, vc, table = paged_case(g, lens, 2, 128, 16, dtype, True)
    table[1, 3] = entry
    q = rand(g, 4, 8, 128, dtype=dtype)
    o, lse = run_paged(q, kc, vc, table, lens, dev)
    with pytest.raises(fm.FMError, match="request 1") as e:
        fm.fm_sync_status()
    assert e.value.code == fm.FM_ERR_INDEX
    ks[1][48:64] = 0
    vs[1][48:64] = 0
    check_paged(q, ks, vs, lens, o, lse)
    fm.fm_sync_status()  # reported once


def test_lengths_that_do_not_fit_are_clamped_and_reported(dev):
    g = torch.Generator(device=dev).manual_seed(16)
    lens = [(1, 100), (1, 64)]
    ks, vs, kc, vc, table = paged_case(g, lens, 2, 128, 16, BF16, True)
    table = table[:, :7].contiguous()  # room for 112 keys
    q = rand(g, 2, 8, 128, dtype=BF16)
    o, lse, ws = torch.empty_like(q), torch.empty(8, 2, device=dev), workspace(2, 2, 8, 2, 128, dev)
    for cu, kv in (([0, 1, 2], [10000, 64]), ([0, 1, 9], [100, 64]), ([0, 1, 0], [100, 64]), ([-5, 1, 2], [100, 64]),
                   ([0, 1, 2], [-3, 64])):
        if kv[0] == 10000:
            table[0] = table[0].clamp(0, kc.shape[0] - 1)
        fm.fm_attn_paged(q, kc, vc, ints(cu, dev), ints(kv, dev), table, fm.seqs_opts(), o, lse, ws)
        with pytest.raises(fm.FMError, match="lengths") as e:
            fm.fm_sync_status()
        assert e.value.code == fm.FM_ERR_INDEX
    # starts that run backwards and so name rows twice
    cu = ints([0, 2, 0, 2], dev)
    fm.fm_attn_varlen(q, q, q, cu, cu, fm.seqs_opts(), o, lse, workspace(3, 2, 8, 8, 128, dev))
    with pytest.raises(fm.FMError):
        fm.fm_sync_status()


# ---------------------------------------------------------------- page tables
class Model:
    """The bookkeeping in plain Python."""

    def __init__(self, n, pages, ps, width):
        self.n, self.ps, self.width, self.pages = n, ps, width, pages
        self.free, self.kv = list(range(pages - 1, -1, -1)), [0] * n
        self.table = [[-1] * width for _ in range(n)]

    def extend(self, new, release, cap):
        up = lambda x: -(-x // self.ps)  # noqa: E731
        base = [0 if r else k for k, r in zip(self.kv, release)]
        free = self.free + [self.table[i][j] for i in range(self.n) if release[i] for j in range(up(self.kv[i]))]
        want = [up(b + x) - up(b) for b, x in zip(base, new)]
        if any(x < 0 for x in new) or any(up(b + x) > self.width for b, x in zip(base, new)) or sum(new) > cap:
            return -1, [0] * (self.n + 1), [-1] * cap, [-1] * cap
        if sum(want) > len(free):
            return sum(want) - len(free), [0] * (self.n + 1), [-1] * cap, [-1] * cap
        slots, pos = [], []
        for i in range(self.n):
            for j in range(want[i]):
                self.table[i][up(base[i]) + j] = free.pop()
            for p in range(base[i], base[i] + new[i]):
                slots.append(self.table[i][p // self.ps] * self.ps + p % self.ps)
                pos.append(p)
            self.kv[i] = base[i] + new[i]
        self.free = free
        fill = [-1] * (cap - len(slots))
        return 0, starts(new), slots + fill, pos + fill


def extend_buffers(n, pages, width, cap, dev, pad=0):
    return dict(kv=ints([0] * n, dev), table=torch.full((n, width + pad), -1, dtype=torch.int32, device=dev)[:, :width],
                free=ints(list(range(pages - 1, -1, -1)), dev), count=ints([pages], dev), cu=ints([9] * (n + 1), dev),
                slots=torch.full((cap,), 9, dtype=torch.int64, device=dev), pos=ints([9] * cap, dev), status=ints([9], dev))


@pytest.mark.parametrize("n,ps,cap,seed", [(1, 1, 7, 0), (5, 16, 300, 1), (40, 3, 5001, 2), (3, 256, 4097, 3), (1100, 8, 20000, 4)])
def test_extend_follows_the_plain_bookkeeping(dev, n, ps, cap, seed):
    """Many steps in place: prompts, single tokens, rows given back and used again in one call,
    calls that are refused for want of pages, table width or slots."""
    r = random.Random(seed)
    width = 40
    pages = max(4, n * 6)
    m, b = Model(n, pages, ps, width), extend_buffers(n, pages, width, cap, dev, pad=3)
    seen = set()
    for step in range(40):
        release = [r.random() < 0.15 and k > 0 for k in m.kv]
        many = r.choice([0.1, 0.5])
        new = [r.choice([0, 1, 1, r.randint(0, 3 * ps) if r.random() < many else 1]) for _ in range(n)]
        if step % 13 == 5:
            new[r.randrange(n)] = r.choice([-1, width * ps + 1, cap + 1, 2 ** 31 - 1])
        if sum(x for x in new if x > 0) > cap and step % 13 != 5:
            new = [min(x, 1) for x in new]
            new = [x if i < cap else 0 for i, x in enumerate(new)]
        status, cu, slots, pos = m.extend(new, release, cap)
        seen.add(min(status, 1))
        rel = ints([int(x) for x in release], dev, torch.uint8) if any(release) or step % 2 else None
        fm.fm_paged_extend(ints(new, dev), rel, b["kv"], b["kv"], b["table"], b["free"], b["count"], b["count"], ps, b["cu"],
                           b["slots"], b["pos"], b["status"])
        assert b["status"].tolist() == [status], (step, status)
        assert b["cu"].tolist() == cu and b["slots"].tolist() == slots and b["pos"].tolist() == pos, step
        assert b["kv"].tolist() == m.kv and b["count"].tolist() == [len(m.free)]
        assert b["free"][:len(m.free)].tolist() == m.free
        for i in range(0, n, max(1, n // 50)):
            held = -(-m.kv[i] // ps)
            assert b["table"][i, :held].tolist() == m.table[i][:held], (step, i)
        if status > 0:  # out of pages: the largest request goes
            big = max(range(n), key=lambda i: m.kv[i])
            release = [i == big for i in range(n)]
            m.extend([0] * n, release, cap)
            fm.fm_paged_extend(ints([0] * n, dev), ints([int(x) for x in release], dev, torch.uint8), b["kv"], b["kv"], b["table"],
                               b["free"], b["count"], b["count"], ps, b["cu"], b["slots"], b["pos"], b["status"])
            assert b["status"].tolist() == [0]
    assert 0 in seen


def test_extend_out_of_place_and_no_requests(dev):
    b = extend_buffers(3, 10, 4, 8, dev)
    kv_out, count_out = ints([7, 7, 7], dev), ints([7], dev)
    call = lambda new, cap=8: fm.fm_paged_extend(ints(new, dev), None, b["kv"], kv_out, b["table"], b["free"], b["count"],  # noqa: E731
                                                 count_out, 4, b["cu"], b["slots"][:cap], b["pos"][:cap], b["status"])
    call([1, 0, 5])
    assert kv_out.tolist() == [1, 0, 5] and count_out.tolist() == [7] and b["kv"].tolist() == [0, 0, 0]
    # the list ends in ... 2, 1, 0: page 0 for the first request, then 1 and 2 for the third
    assert b["slots"].tolist() == [0, 4, 5, 6, 7, 8, -1, -1] and b["pos"].tolist() == [0, 0, 1, 2, 3, 4, -1, -1]
    call([9, 9, 9])  # more tokens than slots: refused, the lengths of the last state are passed on
    assert b["status"].tolist() == [-1] and kv_out.tolist() == [0, 0, 0] and count_out.tolist() == [10]
    call([0, 0, 0], cap=0)
    assert b["status"].tolist() == [0] and b["cu"].tolist() == [0, 0, 0, 0]
    e = extend_buffers(0, 10, 4, 8, dev)
    fm.fm_paged_extend(e["kv"], None, e["kv"], e["kv"], e["table"], e["free"], e["count"], e["count"], 4, e["cu"], e["slots"], e["pos"],
                       e["status"])
    assert e["status"].tolist() == [0] and e["cu"].tolist() == [0] and e["slots"].tolist() == [-1] * 8


# ---------------------------------------------------------------- cache writes
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("H,D,ps,layout", [(2, 128, 16, "token"), (8, 64, 3, "head"), (1, 128, 1, "token"), (3, 64, 128, "odd")])
def test_write_puts_rows_at_their_slots(dev, dtype, H, D, ps, layout):
    g = torch.Generator(device=dev).manual_seed(17)
    pages, T = 9, min(9 * ps - 2, 333)
    kc, vc = (rand(g, pages, ps, H, D + (1 if layout == "odd" else 0), dtype=dtype)[..., :D].transpose(1, 2) for _ in range(2))
    if layout == "head":
        kc, vc = kc.contiguous(), vc.contiguous()
    want_k, want_v = kc.clone(), vc.clone()
    fused = rand(g, T, 2 * H, D, dtype=dtype)
    k, v = fused[:, :H], fused[:, H:]
    slots = torch.randperm(pages * ps, generator=torch.Generator().manual_seed(3))[:T]
    if T > 3:
        slots[[1, T - 1]] = -1
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            want_k[s // ps, :, s % ps], want_v[s // ps, :, s % ps] = k[t], v[t]
    fm.fm_paged_write(k, v, slots.to(dev), kc, vc)
    fm.fm_sync_status()
    assert torch.equal(kc, want_k) and torch.equal(vc, want_v)


def test_write_skips_and_reports_a_slot_outside(dev):
    kc, vc = (torch.zeros(4, 2, 16, 64, dtype=BF16, device=dev) for _ in range(2))
    k = torch.ones(3, 2, 64, dtype=BF16, device=dev)
    fm.fm_paged_write(k, k, ints([5, 64, 6], dev, torch.int64), kc, vc)
    with pytest.raises(fm.FMError, match="token 1") as e:
        fm.fm_sync_status()
    assert e.value.code == fm.FM_ERR_INDEX
    assert float(kc.float().sum()) == float(vc.float().sum()) == 2 * 2 * 64


# ---------------------------------------------------------------- as a server runs them
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("captured", [False, True])
def test_serving_loop(dev, dtype, captured):
    """Prompts in chunks, single tokens, requests that end and rows that are used again, two layers
    with one bookkeeping; every step's attention against each request's whole history.  captured:
    the steps are replays of one graph whose buffers hold up to 96 tokens."""
    g = torch.Generator(device=dev).manual_seed(18)
    n, cap, Hq, Hk, D, ps = 5, 96, 8, 2, 64, 16
    first = fm.PagedKVCache(60, ps, Hk, D, n, 20, cap, dtype=dtype, device=dev)
    layers = [first, fm.PagedKVCache(60, ps, Hk, D, n, 20, cap, dtype=dtype, device=dev, shared=first)]
    for c in layers:
        c.k.fill_(float("nan"))
        c.v.fill_(float("nan"))
    new_d, rel_d = ints([0] * n, dev), ints([0] * n, dev, torch.uint8)
    q, k, v = (torch.zeros(2, cap, h, D, dtype=dtype, device=dev) for h in (Hq, Hk, Hk))
    out = torch.zeros(2, cap, Hq, D, dtype=dtype, device=dev)

    def step():
        first.extend(new_d, rel_d)
        for i, c in enumerate(layers):
            c.write(k[i], v[i])
            c.attention(q[i], out=out[i])

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    if captured:
        with torch.cuda.graph(graph):
            step()
    hist = [[(torch.zeros(0, Hk, D), torch.zeros(0, Hk, D)) for _ in range(2)] for _ in range(n)]
    r = random.Random(2)
    for s in range(14):
        release = [int(s > 3 and r.random() < 0.2) for _ in range(n)]
        new = [r.choice([0, 1, 1, 1, r.randint(1, 30)]) for _ in range(n)]
        while sum(new) > cap:
            new[new.index(max(new))] = 1
        t = sum(new)
        new_d.copy_(ints(new, dev))
        rel_d.copy_(ints(release, dev, torch.uint8))
        for x, h in ((q, Hq), (k, Hk), (v, Hk)):
            x.fill_(float("nan"))  # rows behind the last token are never read
            x[:, :t] = rand(g, 2, t, h, D, dtype=dtype)
        out.fill_(5.0)
        graph.replay() if captured else step()
        fm.fm_sync_status()
        assert first.status.tolist() == [0]
        assert (out[:, t:] == 5.0).all()
        at = 0
        for i in range(n):
            for layer in range(2):
                old = (torch.zeros(0, Hk, D), torch.zeros(0, Hk, D)) if release[i] else hist[i][layer]
                kk = torch.cat([old[0].to(dtype), k[layer, at:at + new[i]].cpu()])
                vv = torch.cat([old[1].to(dtype), v[layer, at:at + new[i]].cpu()])
                hist[i][layer] = (kk, vv)
                if new[i]:
                    ref = attend(q[layer, at:at + new[i]], kk, vv, True, 0, D ** -0.5)
                    assert_close(out[layer, at:at + new[i]], None, *ref, dtype, dtype, D, len(kk))
            at += new[i]
        assert first.kv_len.tolist() == [len(h[0][0]) for h in hist]


def test_a_step_that_does_not_fit_does_nothing(dev):
    c = fm.PagedKVCache(3, 16, 1, 64, 2, 4, 64, dtype=BF16, device=dev)
    c.k.zero_(), c.v.zero_()
    one = torch.ones(64, 1, 64, dtype=BF16, device=dev)
    c.extend(ints([40, 20], dev))
    c.write(one, one)
    o = c.attention(one.clone(), out=torch.full_like(one, 2.0))
    fm.fm_sync_status()
    assert c.status.tolist() == [2] and c.kv_len.tolist() == [0, 0]
    assert not c.k.any() and not c.v.any() and (o == 2.0).all()
    with pytest.raises(fm.FMError):
        c.extend(ints([1], dev))


def test_one_call_form_matches_the_dense_forward(dev):
    """attention_varlen over equal dense requests without a mask is the dense attention forward."""
    g = torch.Generator(device=dev).manual_seed(19)
    B, H, S, D = 2, 3, 200, 128
    q, k, v = (rand(g, B, S, H, D, dtype=F32) for _ in range(3))
    flat = lambda t: t.reshape(B * S, H, D)  # noqa: E731
    cu = ints([0, S, 2 * S], dev)
    o, lse = fm.attention_varlen(flat(q), flat(k), flat(v), cu, causal=False, with_lse=True)
    hsd = lambda t: t.permute(0, 2, 1, 3)  # noqa: E731
    fa = fm.FixedMAttention(B, H, S, S, D, dev)
    dense = fa.forward(hsd(q), hsd(k), hsd(v), with_lse=True)
    fm.fm_sync_status()
    assert float((hsd(o.view(B, S, H, D)) - dense).abs().max()) < 1e-5
    assert float((lse.view(H, B, S).permute(1, 0, 2) - fa.lse).abs().max()) < 1e-5
    assert math.isfinite(float(o.sum()))
