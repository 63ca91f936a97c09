"""The cache's side of drafted trees on the GPU: what is kept of a step's new tokens, the moves of their rows, and whole
decoding loops with drafts."""
import random

import pytest
import torch

import fixed_max_softmax_gb300 as fm
from tests.seqs_reference import assert_close
from tests.test_gpu_guard_bands import Guarded
from tests.test_gpu_seqs import BF16, F16, F32, dev, ints, rand, starts  # noqa: F401
from tests.test_gpu_seqs_guards import Space  # noqa: F401  (the fp16 pattern of Guarded)
from tests.tree_reference import attend_seen, causal_seen, mask_words, random_tree, tree_seen, walk

pytestmark = pytest.mark.gpu


def plain_keep(kv, new, path, kept, table, free, ps, num_pages, width, cols):
    """Lengths, list, moves and status by the header's words, in plain Python; None where the call changes nothing."""
    out, give, src, dst, bad = [], [], [], [], 0
    for i, (s, q) in enumerate(zip(kv, new)):
        k = kept[i]
        p = path[i][:max(k, 0)]
        ok = 0 <= q <= s and -(-s // ps) <= cols and -1 <= k <= min(q, width) and all(a < b for a, b in zip([-1] + p, p)) and all(x < q for x in p)
        bad += not ok
        a, b = [-1] * width, [-1] * width
        n = s
        if ok and k >= 0:
            n = s - q + k
            give += table[i][-(-n // ps):-(-s // ps)]
            slot = lambda x: table[i][x // ps] * ps + x % ps  # noqa: E731, B023
            for j, x in enumerate(p):
                if x != j:
                    a[j], b[j] = slot(s - q + x), slot(s - q + j)
        out.append(n)
        src.append(a)
        dst.append(b)
    return (out, free + give, src, dst, bad) if len(free) + len(give) <= num_pages else None


def keep_case(n, ps, seed, width, bad=False):
    r = random.Random(seed)
    new = [r.choice([0, 1, 2, 9, 33, 64]) for _ in range(n)]
    kv = [q + r.choice([0, 1, ps - 1, ps, 5 * ps + 3, 300]) for q in new]
    cols = max(-(-s // ps) for s in kv) + 2
    pages = sum(-(-s // ps) for s in kv) + 7
    order = list(range(pages))
    r.shuffle(order)
    table = [[order.pop() for _ in range(-(-s // ps))] for s in kv]
    free = order
    kept = [r.choice([-1] + list(range(min(q, width) + 1))) for q in new]
    path = [sorted(r.sample(range(q), max(k, 0))) + [r.randrange(-9, 99) for _ in range(width - max(k, 0))] for q, k in zip(new, kept)]
    if bad:
        for i in range(0, n, 3):
            k = r.randrange(5)
            if k == 0:
                kept[i] = new[i] + 1
            elif k == 1:
                kept[i] = -2
            elif k == 2 and kept[i] > 0:
                path[i][kept[i] - 1] = new[i]
            elif k == 3 and kept[i] > 1:
                path[i][1] = path[i][0]
            elif k == 4 and kept[i] > 0:
                path[i][0] = -1
    return new, kv, cols, pages, table, free, kept, path


@pytest.mark.parametrize("n,ps,width", [(1, 16, 4), (7, 1, 9), (40, 16, 33), (300, 8, 12), (1000, 5, 7), (1500, 16, 8), (3, 128, 64), (8192, 16, 3)])
@pytest.mark.parametrize("bad", [False, True])
@pytest.mark.parametrize("in_place", [True, False])
def test_keep(dev, n, ps, width, bad, in_place):  # noqa: F811
    new, kv, cols, pages, table, free, kept, path = keep_case(n, ps, n + width, width, bad)
    want = plain_keep(kv, new, path, kept, table, free, ps, pages, width, cols)
    g = lambda *shape, dtype=torch.int32: Guarded(shape, dtype, dev)  # noqa: E731
    kv_d, kv_out, lst, count, count_out, status = g(n), g(n), g(pages), g(1), g(1), g(1)
    src, dst = g(2 * n * width), g(2 * n * width)
    kv_d.t.copy_(ints(kv, dev))
    lst.t.copy_(ints(free + [-3] * (pages - len(free)), dev))
    count.t.fill_(len(free))
    tab = Guarded((n, cols), torch.int32, dev, pad=3)
    tab.t.fill_(-5)
    for i, row in enumerate(table):
        if row:
            tab.t[i, :len(row)] = ints(row, dev)
    before = tab.t.clone()
    s64, d64 = (x.t.view(torch.int64).view(n, width) for x in (src, dst))
    out, cout = (kv_d, count) if in_place else (kv_out, count_out)
    fm.fm_paged_keep(ints(starts(new), dev), ints(path, dev), ints(kept, dev), kv_d.t, out.t, tab.t, lst.t, count.t, cout.t, ps,
                     s64, d64, status.t)
    fm.fm_sync_status()
    assert all(x.intact() for x in (kv_d, kv_out, lst, count, count_out, status, src, dst, tab))
    assert out.t.tolist() == want[0] and cout.t.item() == len(want[1]) and status.t.item() == want[4]
    assert lst.t[:len(want[1])].tolist() == want[1] and s64.tolist() == want[2] and d64.tolist() == want[3]
    assert torch.equal(tab.t, before) and (bad or status.t.item() == 0)
    if not in_place:
        assert kv_d.t.tolist() == kv and count.t.item() == len(free)


@pytest.mark.parametrize("count,pages", [(-1, 50), (51, 50), (49, 50)])
def test_a_list_that_does_not_fit_changes_nothing(dev, count, pages):  # noqa: F811
    kv, lst, c = ints([40, 33], dev), ints([7] * pages, dev), ints([count], dev)
    src, dst = (torch.zeros(2, 4, dtype=torch.int64, device=dev) for _ in range(2))
    status, table = ints([5], dev), ints([list(range(5)), list(range(5, 10))], dev)
    fm.fm_paged_keep(ints([0, 20, 40], dev), ints([[0, 1, 2, 3]] * 2, dev), ints([1, 2], dev), kv, kv, table, lst, c, c, 16, src, dst, status)
    fm.fm_sync_status()
    assert kv.tolist() == [40, 33] and c.item() == count and status.item() == -1 and (lst == 7).all()
    assert (src == -1).all() and (dst == -1).all()


def test_lengths_that_cannot_be(dev):  # noqa: F811
    """Starts that run backwards, more new tokens than keys, negative and enormous lengths: such rows stay as they are."""
    i32 = 2 ** 31 - 1
    kv = [10, 5, -3, i32, 40, 10, 100]
    cu = [0, 4, 3, 9, 12, 53, 57, 61]
    c, lst, status = ints([2], dev), ints([0] * 60, dev), ints([9], dev)
    src, dst = (torch.zeros(7, 3, dtype=torch.int64, device=dev) for _ in range(2))
    d = ints(kv, dev)
    table = torch.arange(70, dtype=torch.int32, device=dev).view(7, 10)
    fm.fm_paged_keep(ints(cu, dev), ints([[0, 2, 3]] * 7, dev), ints([2] * 7, dev), d, d, table, lst, c, c, 4, src, dst, status)
    fm.fm_sync_status()
    assert d.tolist() == [8, 5, -3, i32, 40, 8, 100] and status.item() == 5
    assert lst[2:4].tolist() == [2, 52] and c.item() == 4
    assert src[0].tolist() == [-1, 2 * 4 + 0, -1] and dst[0].tolist() == [-1, 1 * 4 + 3, -1]
    assert (src[1:5] == -1).all() and (src[6] == -1).all()


@pytest.mark.parametrize("dtype,D,token_major,ps", [(BF16, 128, True, 16), (F16, 64, False, 8), (F32, 128, True, 5), (BF16, 64, False, 1)])
@pytest.mark.parametrize("odd", [False, True])
def test_moves(dev, dtype, D, token_major, ps, odd):  # noqa: F811
    """Paths of every overlap, caches of both layouts; odd: rows that no 16-byte load takes.  Nothing else changes."""
    g = torch.Generator(device=dev).manual_seed(71)
    n, width, H = 9, 33, 3
    new, kv, cols, pages, table, free, kept, path = keep_case(n, ps, 5, width)
    want = plain_keep(kv, new, path, kept, table, free, ps, pages, width, cols)
    caches, refs = [], []
    for _ in range(2):
        wide = rand(g, *((pages, ps, H, D + 3) if token_major else (pages, H, ps, D + 3)), dtype=dtype)
        full = wide[..., 1:1 + D] if odd else wide[..., :D].contiguous()
        c = full.transpose(1, 2) if token_major else full
        caches.append(c)
        refs.append(c.clone())
    for a, b in zip(want[2], want[3]):
        for x, y in zip(a, b):
            if x >= 0:
                for r in refs:
                    r[y // ps, :, y % ps] = r[x // ps, :, x % ps].clone()
    src, dst = ints(want[2], dev, torch.int64), ints(want[3], dev, torch.int64)
    fm.fm_paged_move(src, dst, *caches)
    fm.fm_sync_status()
    assert all(torch.equal(c, r) for c, r in zip(caches, refs))
    moved = sum(x >= 0 for a in want[2] for x in a)
    assert moved > 20
    # slots past the cache: skipped and reported
    for bad in (src, dst):
        keep, (i, j) = bad.clone(), next((i, j) for i in range(n) for j in range(width) if want[2][i][j] >= 0)
        only = torch.full_like(src, -1)
        a, b = only.clone(), only.clone()
        a[i, j], b[i, j] = src[i, j], dst[i, j]
        (a if bad is src else b)[i, j] = pages * ps
        fm.fm_paged_move(a, b, *caches)
        with pytest.raises(fm.FMError, match="lies outside the cache"):
            fm.fm_sync_status()
        assert all(torch.equal(c, r) for c, r in zip(caches, refs)) and torch.equal(keep, bad)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("dtype,drafted", [(BF16, True), (F32, False)])
def test_decoding_with_drafts(dev, dtype, drafted, captured):  # noqa: F811
    """Prompts, then steps whose new tokens are trees: extend, masks, two layers' writes and attention, verification, the
    kept path moved together; every step's attention against each request's whole history, what is kept against the
    definition, and no page lost.  captured: the steps are replays of one graph."""
    g = torch.Generator(device=dev).manual_seed(72)
    n, cap, Hq, Hk, D, ps, V, width, words = 4, 80, 4, 2, 64, 8, 50, 6, 1
    first = fm.PagedKVCache(80, ps, Hk, D, n, 30, cap, dtype=dtype, device=dev)
    layers = [first, fm.PagedKVCache(80, ps, Hk, D, n, 30, cap, dtype=dtype, device=dev, shared=first)]
    for c in layers:
        c.k.fill_(float("nan"))
        c.v.fill_(float("nan"))
    new_d, rel_d, parent = ints([0] * n, dev), ints([0] * n, dev, torch.uint8), ints([-1] * cap, dev)
    q, k, v = (torch.zeros(2, cap, h, D, dtype=dtype, device=dev) for h in (Hq, Hk, Hk))
    out = torch.zeros(2, cap, Hq, D, dtype=dtype, device=dev)
    lse = torch.zeros(2, Hq, cap, device=dev)
    target, draft = torch.zeros(cap, V, device=dev), torch.zeros(cap, V, device=dev)
    tokens, u, u_last, all_ = ints([0] * cap, dev), torch.zeros(cap, device=dev), torch.zeros(n, device=dev), ints([0] * n, dev)
    seen = {}

    def step():
        first.extend(new_d, rel_d)
        seen["ok"] = first.status.clone()
        mask = first.tree(parent, words)
        for i, c in enumerate(layers):
            c.write(k[i], v[i])
            c.tree_attention(q[i], mask, out=out[i], lse=lse[i])
        path, kept, nxt = fm.verify_tree(target, tokens, parent, first.cu_q, u, u_last, draft if drafted else None, width)
        kept2 = torch.where(all_ != 0, -1, kept)  # prompts keep all they have
        moves = first.keep(path, kept2)
        for c in layers:
            c.move(moves)
        seen.update(mask=mask, path=path, kept=kept, nxt=nxt, status=first.status.clone(), pos=first.positions.clone())

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    if captured:
        with torch.cuda.graph(graph):
            step()
    hist = [[(torch.zeros(0, Hk, D), torch.zeros(0, Hk, D)) for _ in range(2)] for _ in range(n)]
    r = random.Random(4)
    moved = 0
    for s in range(14):
        prompt = [s == 0 or r.random() < 0.15 for _ in range(n)]
        release = [p and s > 0 and r.random() < 0.5 for p in prompt]
        new = [r.choice([0, 3, 33, 38]) if p else r.choice([0, 1, 4, 8, 11]) for p in prompt]
        while sum(new) > cap:
            new[new.index(max(new))] = 5
        prompt = [p and a != 5 for p, a in zip(prompt, new)]
        T = sum(new)
        # (a prompt chunk that fits a mask row is a chain)
        parents = [list(range(-1, a - 1)) if p else random_tree(a, 100 * s + i, 4) for i, (a, p) in enumerate(zip(new, prompt))]
        flat = sum(parents, [])
        for x in (q, k, v):
            x.copy_(rand(g, *x.shape, dtype=dtype))
        target.copy_(torch.softmax(torch.randn(cap, V, generator=g, device=dev) * 2, 1))
        draft.copy_(torch.softmax(torch.log(target) + 0.4 * torch.randn(cap, V, generator=g, device=dev), 1))
        row = [at + max(p, 0) for at, tree in zip(starts(new), parents) for p in tree]  # of each node's parent
        tokens.zero_()
        if T:
            tokens[:T] = torch.multinomial(draft[row], 1, generator=g).flatten().to(torch.int32)
        u.copy_(torch.rand(cap, generator=g, device=dev) * (1.0 if drafted else 0.1))  # (unlikely tokens kept, too)
        u_last.copy_(torch.rand(n, generator=g, device=dev))
        parent.fill_(-1)
        if T:
            parent[:T] = ints(flat, dev)
        new_d.copy_(ints(new, dev))
        rel_d.copy_(ints([int(x) for x in release], dev, torch.uint8))
        all_.copy_(ints([int(x) for x in prompt], dev))
        out.fill_(7.0)
        lse.fill_(7.0)
        if captured:
            graph.replay()
        else:
            step()
        fm.fm_sync_status()
        assert seen["ok"].item() == 0 and seen["status"].item() == 0
        at = starts(new)
        for i in range(n):
            if release[i]:
                hist[i] = [(torch.zeros(0, Hk, D), torch.zeros(0, Hk, D)) for _ in range(2)]
            sl, a = slice(at[i], at[i + 1]), new[i]
            was = hist[i][0][0].shape[0]
            rows_ = mask_words(parents[i], words) if a <= 32 * words else None
            if rows_:
                assert seen["mask"][sl].tolist() == rows_
                see = tree_seen(rows_, was + a)
            else:
                see = causal_seen(a, was + a)
            p, x = walk(target[sl], draft[sl] if drafted else None, tokens[sl].tolist(), parents[i], u[sl].tolist(), float(u_last[i]), width)
            assert seen["path"][i].tolist() == p + [-1] * (width - len(p)) and seen["kept"][i] == len(p) and seen["nxt"][i] == x
            stay = list(range(a)) if prompt[i] else p
            moved += sum(j != y for j, y in enumerate(stay))
            for layer in range(2):
                K, W = (torch.cat([h, t[layer][sl].float().cpu()]) for h, t in zip(hist[i][layer], (k, v)))
                if a:
                    ref = attend_seen(q[layer][sl], K, W, see, D ** -0.5)
                    assert_close(out[layer][sl], lse[layer][:, sl], *ref, dtype, dtype, D, was + a)
                hist[i][layer] = tuple(torch.cat([h, t[layer][sl].float().cpu()[stay]]) for h, t in zip(hist[i][layer], (k, v)))
        assert first.kv_len.tolist() == [h[0][0].shape[0] for h in hist]
        held = [first.block_table[i, :-(-h[0][0].shape[0] // ps)].tolist() for i, h in enumerate(hist)]
        assert sorted(sum(held, []) + first.free_pages[:first.free_count.item()].tolist()) == list(range(80))
        assert (out[:, T:] == 7.0).all()
    assert moved > 10


def test_moves_past_32_bit_offsets(dev):  # noqa: F811
    pages, ps, H, D = 262152, 16, 4, 128
    cache = torch.empty(pages, ps, H, D, dtype=BF16, device=dev).transpose(1, 2)  # 2.1e9 elements
    last, g = pages * ps - 1, torch.Generator(device=dev).manual_seed(73)
    src, dst = [[last, last - 1, 5]], [[3, last - 40, last - 2]]
    rows = rand(g, 3, H, D, dtype=BF16)
    for s, r in zip(src[0], rows):
        cache[s // ps, :, s % ps] = r
    fm.fm_paged_move(ints(src, dev, torch.int64), ints(dst, dev, torch.int64), cache, cache)
    fm.fm_sync_status()
    for s, r in zip(dst[0], rows):
        assert torch.equal(cache[s // ps, :, s % ps], r)


def test_captured_calls_may_be_the_first_of_their_kind(tmp_path):
    """After one attention call on the device every call on trees can be captured though none has run: in a process of
    its own."""
    import subprocess
    import sys

    code = """
import torch, fixed_max_softmax_gb300 as fm
dev = torch.device("cuda:0")
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)
c = {d: fm.PagedKVCache(64, 16, 2, 128, 2, 10, 600, dtype=d, device=dev) for d in (torch.bfloat16, torch.float32)}
first = c[torch.float32]
first.extend(i32([1, 1]))
first.write(torch.ones(2, 2, 128, device=dev), torch.ones(2, 2, 128, device=dev))
first.attention(torch.ones(2, 4, 128, device=dev))
big = fm.PagedKVCache(8, 16, 1, 64, 8192, 1, 16, device=dev)
parent, cu = i32([-1, 0, 0, 1] * 2), None
p = {d: torch.full((8, 1000), 1e-3, dtype=d, device=dev) for d in (torch.float32, torch.bfloat16, torch.float16)}
u, last, tok, new = torch.full((8,), .5, device=dev), torch.full((2,), .5, device=dev), i32([1] * 8), i32([4, 4])
wide, none = torch.zeros(8192, 2, dtype=torch.int32, device=dev), torch.zeros(8192, dtype=torch.int32, device=dev)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    for d, x in c.items():
        x.extend(new)
        m = x.tree(parent, 1)
        rows = torch.ones(8, 2, 128, dtype=d, device=dev)
        x.write(rows, rows)
        o = x.tree_attention(torch.ones(8, 4, 128, dtype=d, device=dev), m)
        for q in p.values():
            for draft in (None, q):
                path, kept, nxt = fm.verify_tree(q, tok, parent, x.cu_q, u, last, draft, 4)
        x.move(x.keep(path, kept))
    big.move(big.keep(wide, none))
g.replay()
fm.fm_sync_status()
assert ((o - 1).abs() <= 2 * (5 + 8) * 2.0 ** -24).all() and kept.tolist() == [3, 3] and nxt.tolist() == [500, 500], (o, kept, nxt)
assert c[torch.bfloat16].kv_len.tolist() == [3, 3] and big.kv_len.sum() == 0
print("captured")
"""
    path = tmp_path / "first.py"
    path.write_text(code)
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, str(path)], capture_output=True, text=True, timeout=300, env=dict(os.environ, PYTHONPATH=root))
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]
