"""Verification of trees of drafted tokens on the GPU against the definition in 64 bits (tests/tree_reference.py): the
same nodes, the same next token.  Sums and products are the definition's to some 2^-45, random numbers have 24 bits."""
import math

import pytest
import torch

import fixed_max_softmax_gb300 as fm
from tests.test_gpu_guard_bands import Guarded
from tests.test_gpu_seqs import BF16, F16, F32, dev, ints, starts  # noqa: F401
from tests.tree_reference import random_tree, walk

pytestmark = pytest.mark.gpu


def tree_case(g, counts, V, dtype, drafted, shape="tree", sharp=4.0):
    """Rows of a target and of a draft near it, trees, tokens drawn from the draft's rows (or its likeliest)."""
    T = sum(counts)
    logits = torch.randn(T, V, generator=g, device=g.device) * 1.5
    hot = torch.randint(0, V, (T, 6), generator=g, device=g.device)
    logits.scatter_add_(1, hot, torch.randn(T, 6, generator=g, device=g.device) + sharp + math.log(V) / 2)
    target = torch.softmax(logits, 1).to(dtype)
    draft = torch.softmax(logits + torch.randn(T, V, generator=g, device=g.device) * 0.7, 1).to(dtype)
    parents, tokens, at = [], [], 0
    for i, n in enumerate(counts):
        p = list(range(-1, n - 1)) if shape == "chain" else random_tree(n, 900 + i) if shape == "tree" else ([-1] + [0] * (n - 1))[:n]
        toks = [0] * n
        for node in set(p) - {-1}:
            kids = [t for t in range(n) if p[t] == node]
            row = draft[at + node].float()
            guess = torch.multinomial(row, len(kids), True, generator=g) if drafted else row.topk(min(V, len(kids))).indices
            for j, t in enumerate(kids):
                toks[t] = int(guess[min(j, len(guess) - 1)])
        parents += p
        tokens += toks
        at += n
    u, u_last = (torch.rand(m, generator=g, device=g.device) for m in (T, len(counts)))
    return target, draft if drafted else None, tokens, parents, u, u_last


def verify(target, draft, counts, tokens, parents, u, u_last, dev, max_path=12, cu=None):  # noqa: F811
    n, T = len(counts), len(tokens)
    target, draft = target[:T], None if draft is None else draft[:T]
    path = Guarded((n, max_path), torch.int32, dev)
    kept, nxt = Guarded((n,), torch.int32, dev), Guarded((n,), torch.int32, dev)
    for x in (path, kept, nxt):
        x.t.fill_(-7)
    fm.fm_tree_verify(target, draft, cu if cu is not None else ints(starts(counts), dev), ints(tokens, dev), ints(parents, dev), u, u_last,
                      path.t, kept.t, nxt.t)
    return path, kept, nxt


def check(target, draft, counts, tokens, parents, u, u_last, max_path, got):
    assert all(x.intact() for x in got)
    path, kept, nxt = (x.t.tolist() for x in got)
    at = starts(counts)
    for i in range(len(counts)):
        sl = slice(at[i], at[i + 1])
        p, x = walk(target[sl], None if draft is None else draft[sl], tokens[sl], parents[sl], u[sl].tolist(), float(u_last[i]), max_path)
        assert path[i] == p + [-1] * (max_path - len(p)) and kept[i] == len(p) and nxt[i] == x, i


@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 1000, 4099, 50021])
@pytest.mark.parametrize("shape", ["tree", "chain", "star"])
def test_verify(dev, shape, V, dtype, drafted):  # noqa: F811
    g = torch.Generator(device=dev).manual_seed(60)
    counts = [9, 1, 0, 26, 2, 5, 17]
    c = tree_case(g, counts, V, dtype, drafted, shape)
    got = verify(c[0], c[1], counts, *c[2:], dev)
    fm.fm_sync_status()
    check(c[0], c[1], counts, *c[2:], 12, got)


@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("n,V", [(1, 128000), (30, 20000), (60, 9001), (90, 5000), (160, 3001), (400, 600)])
def test_clusters_of_every_size(dev, n, V, drafted):  # noqa: F811
    g = torch.Generator(device=dev).manual_seed(61)
    counts = [1 + (i * 5) % 12 for i in range(n)]
    c = tree_case(g, counts, V, F32, drafted)
    got = verify(c[0], c[1], counts, *c[2:], dev)
    again = verify(c[0], c[1], counts, *c[2:], dev)
    fm.fm_sync_status()
    check(c[0], c[1], counts, *c[2:], 12, got)
    assert all(torch.equal(a.t, b.t) for a, b in zip(got, again))


@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("dtype,offset,q_offset,pad", [(F32, 1, 1, 0), (F32, 3, 2, 5), (BF16, 5, 5, 3), (F16, 7, 1, 2), (BF16, 8, 0, 8)])
def test_rows_of_any_alignment(dev, dtype, offset, q_offset, pad, drafted):  # noqa: F811
    """Rows as parts of wider ones whose other elements are NaN; the draft's aligned otherwise than the target's."""
    g = torch.Generator(device=dev).manual_seed(62)
    counts, V = [9, 20, 3], 2305
    c = tree_case(g, counts, V, dtype, drafted)

    def inside(x, off):
        if x is None:
            return None
        wide = torch.full((x.shape[0], V + off + pad), float("nan"), dtype=dtype, device=dev)
        wide[:, off:off + V] = x
        return wide[:, off:off + V]

    p, q = inside(c[0], offset), inside(c[1], q_offset)
    got = verify(p, q, counts, *c[2:], dev)
    fm.fm_sync_status()
    check(p, q, counts, *c[2:], 12, got)


@pytest.mark.parametrize("drafted", [True, False])
@pytest.mark.parametrize("max_path", [1, 2, 3, 40])
def test_paths_of_limited_length(dev, max_path, drafted):  # noqa: F811
    g = torch.Generator(device=dev).manual_seed(63)
    counts = [30] * 12
    c = tree_case(g, counts, 500, F32, drafted, "chain", sharp=9.0)
    c[4].mul_(0.2)
    got = verify(c[0], c[1], counts, *c[2:], dev, max_path)
    fm.fm_sync_status()
    check(c[0], c[1], counts, *c[2:], max_path, got)
    assert max_path > 30 or got[1].t.max() == max_path


@pytest.mark.parametrize("drafted", [True, False])
def test_large_trees(dev, drafted):  # noqa: F811
    """1,024 nodes, hundreds of them children of one node; a chain that is kept to its end."""
    g = torch.Generator(device=dev).manual_seed(64)
    for shape, counts in (("star", [1024, 300]), ("tree", [1024, 1000])):
        c = tree_case(g, counts, 300, F32, drafted, shape, sharp=0.0)
        got = verify(c[0], c[1], counts, *c[2:], dev, 1024)
        fm.fm_sync_status()
        check(c[0], c[1], counts, *c[2:], 1024, got)
    p = torch.zeros(1024, 8, device=dev)
    p[:, 5] = 1.0
    got = verify(p, p if drafted else None, [1024], [5] * 1024, list(range(-1, 1023)), torch.rand(1024, generator=g, device=dev),
                 torch.zeros(1, device=dev), dev, 1024)
    assert got[0].t[0].tolist() == list(range(1024)) and got[1].t.item() == 1024 and got[2].t.item() == 5


@pytest.mark.parametrize("drafted", [True, False])
def test_distributions_that_are_none(dev, drafted):  # noqa: F811
    """Rows of zeros, single tokens, infinities, NaN, negative numbers; numbers outside [0, 1); children of one token."""
    g = torch.Generator(device=dev).manual_seed(65)
    V, n = 40, 64
    counts = [8] * n
    target, draft, tokens, parents, u, u_last = tree_case(g, counts, V, F32, drafted, "tree", sharp=0.0)
    odd = torch.tensor([0.0, -1.0, float("nan"), float("inf"), -float("inf"), 1e-42, 1e-30], device=dev)
    for x in [target] + ([draft] if drafted else []):
        where = torch.rand(x.shape, generator=g, device=dev)
        put = odd[torch.randint(0, 7, x.shape, generator=g, device=dev)]
        x[: 8 * n // 2] = torch.where(where[: 8 * n // 2] < 0.3, put[: 8 * n // 2], x[: 8 * n // 2])
        x[40:60] = 0.0
        x[60:90] = 0.0
        x[60:90, 3] = 1.0
    tokens = [3 if i % 3 == 0 else t for i, t in enumerate(tokens)]
    strange = torch.tensor([0.0, 1.0, 1.5, -1.0, float("nan"), 0.5, 2.0 ** -24, 1 - 2.0 ** -24], device=dev)
    u[::2] = strange[torch.randint(0, 8, u[::2].shape, generator=g, device=dev)]
    u_last[::2] = strange[torch.randint(0, 8, u_last[::2].shape, generator=g, device=dev)]
    got = verify(target, draft, counts, tokens, parents, u, u_last, dev)
    fm.fm_sync_status()
    check(target, draft, counts, tokens, parents, u, u_last, 12, got)
    assert (got[2].t == -1).any()


def test_tokens_outside_and_too_many_nodes_are_reported(dev):  # noqa: F811
    p = torch.full((1100, 16), 1 / 16, device=dev)
    u, last = torch.zeros(1100, device=dev), torch.full((3,), 0.99, device=dev)
    for bad in (16, -1, 2 ** 31 - 1, -2 ** 31):
        got = verify(p, p, [3], [0, bad, 4], [-1, 0, 0], u[:3], last, dev)
        with pytest.raises(fm.FMError, match="token of node 1") as e:
            fm.fm_sync_status()
        assert e.value.code == fm.FM_ERR_INDEX
        assert got[0].t[0, :3].tolist() == [0, 2, -1] and got[2].t.item() == 15
    # (node 0's own token is looked at nowhere)
    got = verify(p, p, [2], [-5, 4], [-1, 0], u[:2], last, dev)
    fm.fm_sync_status()
    assert got[1].t.item() == 2
    got = verify(p, None, [3, 1025, 2], [0] * 1030, [-1, 0, 0] + list(range(-1, 1024)) + [-1, 0], u[:1030], last, dev)
    with pytest.raises(fm.FMError, match="do not fit"):
        fm.fm_sync_status()
    assert got[1].t.tolist() == [2, 0, 2] and got[2].t.tolist() == [15, -1, 15] and (got[0].t[1] == -1).all()
    for cu in ([0, 3, 5000], [0, -5, 3], [7, 2, 6]):
        got = verify(p, None, [0, 0], [0] * 1100, [-1] * 1100, u, last, dev, cu=ints(cu, dev))
        with pytest.raises(fm.FMError, match="do not fit"):
            fm.fm_sync_status()
        assert all(x.intact() for x in got)
    # parents that are no earlier node: such nodes are never tried
    got = verify(p, p, [5], [1] * 5, [-1, 1, 7, -9, 0], u[:5], last, dev)
    fm.fm_sync_status()
    assert got[0].t[0, :3].tolist() == [0, 4, -1]


def test_one_row_for_every_node_and_two_calls_at_once(dev):  # noqa: F811
    """Rows 0 elements apart; two streams."""
    g = torch.Generator(device=dev).manual_seed(66)
    counts, V = [12] * 20, 30011
    base = torch.softmax(torch.randn(1, V, generator=g, device=dev) * 3, 1)
    p = base.expand(240, V)
    c = tree_case(g, counts, V, F32, True)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    with torch.cuda.stream(s[0]):
        a = verify(p, p, counts, *c[2:], dev)
    with torch.cuda.stream(s[1]):
        b = verify(c[0], c[1], counts, *c[2:], dev)
    torch.cuda.synchronize()
    fm.fm_sync_status()
    check(p, p, counts, *c[2:], 12, a)
    check(c[0], c[1], counts, *c[2:], 12, b)


def test_verify_captured_and_replayed(dev):  # noqa: F811
    g = torch.Generator(device=dev).manual_seed(67)
    room, V, n = 40, 7001, 4
    bufs = tree_case(g, [10] * 4, V, BF16, True)
    target, draft, u, u_last = bufs[0], bufs[1], bufs[4], bufs[5]
    cu, tokens, parents = ints([0] * 5, dev), ints([0] * room, dev), ints([-1] * room, dev)
    path, kept, nxt = ints([[0] * 6] * n, dev), ints([0] * n, dev), ints([0] * n, dev)
    call = lambda: fm.fm_tree_verify(target, draft, cu, tokens, parents, u, u_last, path, kept, nxt)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for counts in ([10] * 4, [1, 0, 30, 9], [0, 0, 0, 0]):
        c = tree_case(g, counts, V, BF16, True)
        T = sum(counts)
        for dst, src in ((target, c[0]), (draft, c[1]), (u, c[4])):
            dst[:T] = src
        u_last.copy_(c[5])
        tokens[:T], parents[:T] = ints(c[2], dev), ints(c[3], dev)
        cu.copy_(ints(starts(counts), dev))
        graph.replay()
        fm.fm_sync_status()
        at = starts(counts)
        for i in range(n):
            sl = slice(at[i], at[i + 1])
            p, x = walk(c[0][sl], c[1][sl], c[2][sl], c[3][sl], c[4][sl].tolist(), float(u_last[i]), 6)
            assert path[i].tolist() == p + [-1] * (6 - len(p)) and kept[i] == len(p) and nxt[i] == x


@pytest.mark.parametrize("drafted", [True, False])
def test_rows_past_32_bit_offsets(dev, drafted):  # noqa: F811
    """The last rows of 20,000 by 131,072."""
    g = torch.Generator(device=dev).manual_seed(68)
    T, V, counts = 20000, 131072, [9, 7]
    c = tree_case(g, counts, V, BF16, drafted)
    far = [torch.empty(T, V, dtype=BF16, device=dev) for _ in range(2 if drafted else 1)]
    for x, y in zip(far, c[:2]):
        x[-16:] = y
    pad = lambda x: torch.cat([torch.zeros(T - 16, dtype=x.dtype, device=dev), x])  # noqa: E731
    path, kept, nxt = ints([[0] * 8] * 2, dev), ints([0] * 2, dev), ints([0] * 2, dev)
    fm.fm_tree_verify(far[0], far[1] if drafted else None, ints([T - 16, T - 7, T], dev), pad(ints(c[2], dev)), pad(ints(c[3], dev)),
                      pad(c[4]), c[5], path, kept, nxt)
    fm.fm_sync_status()
    for i, sl in enumerate((slice(0, 9), slice(9, 16))):
        p, x = walk(c[0][sl], c[1][sl] if drafted else None, c[2][sl], c[3][sl], c[4][sl].tolist(), float(c[5][i]), 8)
        assert path[i].tolist() == p + [-1] * (8 - len(p)) and kept[i] == len(p) and nxt[i] == x
