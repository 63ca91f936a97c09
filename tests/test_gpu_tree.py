"""Attention of trees of drafted tokens over the paged cache and their masks, on the GPU, against plain 64-bit
computations (bounds as for the other serving calls: tests/seqs_reference.py)."""
import random

import pytest
import torch

import fixed_max_softmax_gb300 as fm
from tests.seqs_reference import assert_close
from tests.test_gpu_seqs import BF16, F16, F32, dev, ints, paged_case, rand, run_paged, starts, workspace  # noqa: F401
from tests.test_gpu_seqs_guards import Space  # (also the fp16 pattern of Guarded)
from tests.test_gpu_guard_bands import Guarded
from tests.tree_reference import ancestors, attend_seen, causal_seen, mask_words, random_tree, tree_seen

pytestmark = pytest.mark.gpu


def trees_of(lens, words, seed=5):
    """Parents of each request (None: too many tokens for a mask row, causal)."""
    return [random_tree(a, seed + i) if a <= 32 * words else None for i, (a, _) in enumerate(lens)]


def mask_of(parents, lens, words, dev):  # noqa: F811
    rows = []
    for p, (a, _) in zip(parents, lens):
        rows += mask_words(p, words) if p is not None else [[0x55555555] * words] * a  # (not looked at)
    return torch.tensor(rows or [[0] * words], dtype=torch.int32, device=dev)[: sum(a for a, _ in lens)]


def run_tree(q, kc, vc, table, lens, mask, dev, out_dtype=None, scale=0.0):  # noqa: F811
    T, Hq, D = q.shape
    o = torch.full((T, Hq, D), 7.0, dtype=out_dtype or q.dtype, device=dev)
    lse = torch.full((Hq, T), 7.0, device=dev)
    fm.fm_attn_tree(q, kc, vc, ints(starts([a for a, _ in lens]), dev), ints([b for _, b in lens], dev), table, mask,
                    fm.seqs_opts(softmax_scale=scale), o, lse, workspace(len(lens), T, Hq, kc.shape[1], D, dev))
    return o, lse


def check_tree(q, ks, vs, lens, mask, words, o, lse, scale=0.0):
    D, at = q.shape[2], starts([a for a, _ in lens])
    rows = mask.cpu().tolist()
    for i, (a, b) in enumerate(lens):
        sl = slice(at[i], at[i + 1])
        seen = tree_seen(rows[sl], b) if 0 < a <= 32 * words else causal_seen(a, b)
        assert_close(o[sl], lse[:, sl], *attend_seen(q[sl], ks[i], vs[i], seen, scale or D ** -0.5), q.dtype, o.dtype, D, b)


LENS = {
    "one node": [(1, 1), (1, 300), (1, 0)],
    "small": [(5, 5), (9, 130), (2, 2), (0, 7), (0, 0), (26, 600)],
    "borders": [(32, 160), (31, 158), (33, 161), (8, 128), (8, 129), (8, 135), (8, 136), (64, 64)],
    "large trees": [(70, 333), (130, 1000), (250, 250)],
    "chunks beside": [(300, 700), (7, 90), (1, 1), (257, 257), (40, 1999)],
    "more nodes than keys": [(20, 7), (9, 0), (12, 12)],
    "long": [(12, 5000), (3, 9000)],
    "many": [(3, 40)] * 150 + [(16, 333)],
}


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (F16, 128), (BF16, 64), (F16, 64), (F32, 128), (F32, 64)])
@pytest.mark.parametrize("name", list(LENS))
def test_tree_lengths(dev, name, dtype, D):  # noqa: F811
    g = torch.Generator(device=dev).manual_seed(41)
    lens, words = LENS[name], 8
    ks, vs, kc, vc, table = paged_case(g, lens, 2, D, 16, dtype, True)
    q = rand(g, sum(a for a, _ in lens), 6, D, dtype=dtype, scale=1.5)
    mask = mask_of(trees_of(lens, words), lens, words, dev)
    o, lse = run_tree(q, kc, vc, table, lens, mask, dev)
    fm.fm_sync_status()
    check_tree(q, ks, vs, lens, mask, words, o, lse)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (5, 1), (7, 7), (14, 2), (24, 3), (32, 1), (64, 1)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_tree_heads(dev, Hq, Hk, dtype):  # noqa: F811
    g = torch.Generator(device=dev).manual_seed(42)
    lens, words = [(17, 300), (1, 40), (33, 129)], 2
    ks, vs, kc, vc, table = paged_case(g, lens, Hk, 128, 16, dtype, False)
    q = rand(g, 51, Hq, 128, dtype=dtype)
    mask = mask_of(trees_of(lens, words), lens, words, dev)
    o, lse = run_tree(q, kc, vc, table, lens, mask, dev)
    fm.fm_sync_status()
    check_tree(q, ks, vs, lens, mask, words, o, lse)


@pytest.mark.parametrize("ps", [1, 5, 8, 16, 24, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype,D,out", [(BF16, 128, BF16), (F16, 64, F32), (F32, 64, F32)])
def test_tree_page_sizes_and_layouts(dev, ps, dtype, D, out):  # noqa: F811
    g = torch.Generator(device=dev).manual_seed(43)
    lens, words = [(20, 400), (31, 31), (6, 131), (90, 200)], 3
    ks, vs, kc, vc, table = paged_case(g, lens, 2, D, ps, dtype, ps % 2 == 0)
    q = rand(g, 147, 2 + 6, D, dtype=dtype)[:, 2:]
    wide = torch.full((147, words + 3), -1, dtype=torch.int32, device=dev)  # a mask inside a wider array
    wide[:, 1:1 + words] = mask_of(trees_of(lens, words), lens, words, dev)
    mask = wide[:, 1:1 + words]
    o, lse = run_tree(q, kc, vc, table, lens, mask, dev, out)
    fm.fm_sync_status()
    check_tree(q, ks, vs, lens, mask, words, o, lse)


@pytest.mark.parametrize("dtype,Hk", [(BF16, 2), (F32, 2), (BF16, 8), (F32, 8)])
@pytest.mark.parametrize("words", [1, 2, 5])
def test_any_mask(dev, dtype, Hk, words):  # noqa: F811
    """Random bits (those of later tokens and of tokens that the request does not have are not looked at), rows of zeros,
    rows that see nothing at all."""
    g = torch.Generator(device=dev).manual_seed(44)
    lens = [(32, 32), (30, 500), (3, 3), (25, 130), (32, 1000)]
    ks, vs, kc, vc, table = paged_case(g, lens, Hk, 128, 16, dtype, True)
    T = sum(a for a, _ in lens)
    q = rand(g, T, 8, 128, dtype=dtype)
    mask = torch.randint(-2 ** 31, 2 ** 31, (T, words), generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    mask[::5] = 0
    o, lse = run_tree(q, kc, vc, table, lens, mask, dev)
    fm.fm_sync_status()
    check_tree(q, ks, vs, lens, mask, words, o, lse)
    assert (o[0] == 0).all() and torch.isneginf(lse[:, 0]).all()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("lens", [[(25, 900)] * 24, [(1, 2600)] * 20, [(40, 4000), (8, 500), (9, 9)] * 6,
                                  ([(70, 900)] + [(1, 5)] * 9) * 6, [(5, 700)] * 90])
def test_a_chain_is_causal(dev, dtype, lens):  # noqa: F811
    """Trees without a branch are causal attention, and give fm_attn_paged's bits where both cut their work alike (at most
    128 rows a request, and work for the whole GPU)."""
    g = torch.Generator(device=dev).manual_seed(45)
    ks, vs, kc, vc, table = paged_case(g, lens, 2, 128, 16, dtype, True)
    q = rand(g, sum(a for a, _ in lens), 10, 128, dtype=dtype)
    words = 2
    mask = mask_of([list(range(-1, a - 1)) if a <= 32 * words else None for a, _ in lens], lens, words, dev)
    o, lse = run_tree(q, kc, vc, table, lens, mask, dev)
    o2, lse2 = run_paged(q, kc, vc, table, lens, dev)
    fm.fm_sync_status()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    at = starts([a for a, _ in lens])
    for i in range(0, len(lens), max(1, len(lens) // 12)):
        (a, b), sl = lens[i], slice(at[i], at[i + 1])
        ref = attend_seen(q[sl], ks[i], vs[i], causal_seen(a, b), 128 ** -0.5)
        assert_close(o[sl], lse[:, sl], *ref, dtype, dtype, 128, b)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_the_largest_tree(dev, dtype):  # noqa: F811
    g = torch.Generator(device=dev).manual_seed(46)
    lens, words = [(1024, 1100), (2, 70)], 32
    ks, vs, kc, vc, table = paged_case(g, lens, 1, 64, 64, dtype, True)
    q = rand(g, 1026, 2, 64, dtype=dtype)
    parents = trees_of(lens, words)
    mask, pos = torch.zeros(1026, words, dtype=torch.int32, device=dev), torch.zeros(1026, dtype=torch.int32, device=dev)
    fm.fm_tree_mask(ints(sum(parents, []), dev), ints([0, 1024, 1026], dev), ints([1100, 70], dev), mask, pos)
    assert torch.equal(mask, mask_of(parents, lens, words, dev))
    o, lse = run_tree(q, kc, vc, table, lens, mask, dev)
    fm.fm_sync_status()
    at = [0, 1024, 1026]
    for i, (a, b) in enumerate(lens):
        seen = torch.ones(a, b, dtype=torch.bool)
        for t, s in enumerate(ancestors(parents[i])):
            seen[t, b - a:] = False
            seen[t, [b - a + j for j in s]] = True
        sl = slice(at[i], at[i + 1])
        assert_close(o[sl], lse[:, sl], *attend_seen(q[sl], ks[i], vs[i], seen, 64 ** -0.5), dtype, dtype, 64, b)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("name", ["small", "chunks beside", "long"])
def test_tree_stays_inside(dev, dtype, name):  # noqa: F811
    """Nothing outside the outputs and the workspace is written; rows behind the last request are left as they were."""
    g = torch.Generator(device=dev).manual_seed(47)
    lens, words = LENS[name], 2
    ks, vs, kc, vc, table = paged_case(g, lens, 2, 128, 16, dtype, True)
    T = sum(a for a, _ in lens)
    q = rand(g, T + 5, 8, 128, dtype=dtype)
    o, lse = Guarded((T + 5, 8, 128), dtype, dev, pad=32), Guarded((8, T + 5), F32, dev)
    o.t.fill_(3.0)
    lse.t.fill_(3.0)
    ws = Space(fm.fm_attn_seqs_workspace_size(len(lens), T + 5, 8, 2, 128), dev)
    mask = torch.cat([mask_of(trees_of(lens, words), lens, words, dev), ints([[-1] * words] * 5, dev)])
    fm.fm_attn_tree(q, kc, vc, ints(starts([a for a, _ in lens]), dev), ints([b for _, b in lens], dev), table, mask,
                    fm.seqs_opts(), o.t, lse.t, ws.t)
    fm.fm_sync_status()
    assert o.intact() and lse.intact() and ws.intact()
    assert (o.t[T:] == 3.0).all() and (lse.t[:, T:] == 3.0).all()
    check_tree(q[:T], ks, vs, lens, mask[:T], words, o.t[:T], lse.t[:, :T])


def test_tree_captured_and_replayed_with_other_lengths_and_trees(dev):  # noqa: F811
    g = torch.Generator(device=dev).manual_seed(48)
    n, room, words = 3, 40, 1
    ks, vs, kc, vc, table = paged_case(g, [(0, 500), (0, 1300), (0, 40)], 2, 128, 16, BF16, True)
    q = rand(g, room, 8, 128, dtype=BF16)
    o, lse = torch.empty_like(q), torch.empty(8, room, device=dev)
    cu, kv, parent = ints([0, 1, 2, 3], dev), ints([5, 5, 5], dev), ints([-1] * room, dev)
    mask, pos = torch.zeros(room, words, dtype=torch.int32, device=dev), torch.zeros(room, dtype=torch.int32, device=dev)
    ws, opt = workspace(n, room, 8, 2, 128, dev), fm.seqs_opts()

    def step():
        fm.fm_tree_mask(parent, cu, kv, mask, pos)
        fm.fm_attn_tree(q, kc, vc, cu, kv, table, mask, opt, o, lse, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed, lens in enumerate(([(10, 500), (20, 1300), (10, 40)], [(1, 1), (7, 7), (0, 0)], [(32, 300), (0, 3), (8, 33)])):
        parents = [random_tree(a, 70 + seed + i) if a else [] for i, (a, _) in enumerate(lens)]
        flat = sum(parents, [])
        cu.copy_(ints(starts([a for a, _ in lens]), dev))
        kv.copy_(ints([b for _, b in lens], dev))
        parent[:len(flat)] = ints(flat, dev)
        graph.replay()
        fm.fm_sync_status()
        T = len(flat)
        check_tree(q[:T], [k[:b] for k, (_, b) in zip(ks, lens)], [v[:b] for v, (_, b) in zip(vs, lens)], lens, mask[:T], words,
                   o[:T], lse[:, :T])


def test_two_tree_calls_at_once(dev):  # noqa: F811
    """Two streams with a workspace each, and the same bits every time."""
    g = torch.Generator(device=dev).manual_seed(49)
    lens, words = [(9, 3000)] * 6, 1
    cases = [paged_case(g, lens, 2, 128, 16, BF16, True) for _ in range(2)]
    q = [rand(g, 54, 8, 128, dtype=BF16) for _ in range(2)]
    mask = mask_of(trees_of(lens, words), lens, words, dev)
    torch.cuda.synchronize()
    streams, outs, first = [torch.cuda.Stream(), torch.cuda.Stream()], [None, None], None
    for _ in range(3):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                outs[i] = run_tree(q[i], c[2], c[3], c[4], lens, mask, dev)
        torch.cuda.synchronize()
        first = first or [x.clone() for x, _ in outs]
        assert all(torch.equal(a, b) for a, (b, _) in zip(first, outs))
    fm.fm_sync_status()
    for i, c in enumerate(cases):
        check_tree(q[i], c[0], c[1], lens, mask, words, *outs[i])


# ---------------------------------------------------------------- masks
@pytest.mark.parametrize("words", [1, 2, 3, 8])
@pytest.mark.parametrize("seed", range(4))
def test_masks_and_positions(dev, words, seed):  # noqa: F811
    """Trees of all sizes and shapes (chains, stars, forests), prompt chunks beside them, requests without tokens; a
    mask inside a wider array, rows behind the last request."""
    r = random.Random(seed)
    lens = [(r.choice([0, 1, 2, 31, 32, 33, 64, 65, 96, 32 * words, 32 * words + 1, 300]), r.randrange(0, 5000)) for _ in range(40)]
    lens = [(a, max(a, b)) for a, b in lens]
    parents = []
    for i, (a, _) in enumerate(lens):
        kind = r.randrange(4)
        p = [list(range(-1, a - 1)), [-1] + [0] * (a - 1), [t - 1 if r.random() < 0.8 else -1 for t in range(a)], random_tree(a, i, 50)][kind]
        parents.append(p[:a])
    T, extra = sum(a for a, _ in lens), 4
    flat = sum((p if a <= 32 * words else [99] * a for p, (a, _) in zip(parents, lens)), []) + [77] * extra
    wide = Guarded((T + extra, words), torch.int32, dev, pad=2)
    pos = Guarded((T + extra,), torch.int32, dev)
    wide.t.fill_(123)
    pos.t.fill_(123)
    fm.fm_tree_mask(ints(flat, dev), ints(starts([a for a, _ in lens]), dev), ints([b for _, b in lens], dev), wide.t, pos.t)
    fm.fm_sync_status()
    assert wide.intact() and pos.intact()
    want, at = [], []
    for p, (a, b) in zip(parents, lens):
        if a > 32 * words:
            want += [[0] * words] * a
            at += range(b - a, b)
        elif a:
            want += mask_words(p, words)
            at += [b - a + len(s) - 1 for s in ancestors(p)]
    assert wide.t[:T].tolist() == want and pos.t[:T].tolist() == at
    assert (wide.t[T:] == 123).all() and (pos.t[T:] == 123).all()
    again = torch.full((T + extra, words), 5, dtype=torch.int32, device=dev)
    fm.fm_tree_mask(ints(flat, dev), ints(starts([a for a, _ in lens]), dev), ints([b for _, b in lens], dev), again)
    assert torch.equal(again[:T], wide.t[:T])


def test_bad_parents_and_starts_are_reported(dev):  # noqa: F811
    mask, pos = torch.zeros(6, 1, dtype=torch.int32, device=dev), torch.zeros(6, dtype=torch.int32, device=dev)
    kv = ints([10, 10], dev)
    for bad in (3, 4, 5, 2 ** 31 - 1, -2, -2 ** 31):
        fm.fm_tree_mask(ints([-1, 0, 1, bad, 0, 1], dev), ints([0, 6, 6], dev), kv, mask, pos)
        with pytest.raises(fm.FMError, match="parent of node 3") as e:
            fm.fm_sync_status()
        assert e.value.code == fm.FM_ERR_INDEX
        assert mask.flatten().tolist() == [1, 3, 7, 8, 17, 35] and pos.tolist() == [4, 5, 6, 4, 5, 6]
    fm.fm_sync_status()
    for cu in ([0, 3, 9], [0, -5, 3], [5, 2, 6], [-2, 1, 2]):
        fm.fm_tree_mask(ints([-1] * 6, dev), ints(cu, dev), kv, mask, pos)
        with pytest.raises(fm.FMError, match="do not fit"):
            fm.fm_sync_status()
