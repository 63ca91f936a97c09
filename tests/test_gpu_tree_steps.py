"""Steps with drafted tokens through PagedKVCache and verify_tree() as a program makes them, where parts of a step go
wrong or are not trees."""
import random

import pytest
import torch

import fixed_max_softmax_gb300 as fm
from tests.seqs_reference import assert_close
from tests.test_gpu_guard_bands import Guarded
from tests.test_gpu_seqs import BF16, F16, F32, dev, ints, rand, starts  # noqa: F401
from tests.test_gpu_tree_verify import tree_case
from tests.tree_reference import attend_seen, causal_seen, mask_words, random_tree, tree_seen, walk

pytestmark = pytest.mark.gpu


def test_a_path_buffer_with_more_rows_than_the_cache(dev):  # noqa: F811
    """Only the cache's rows move, whatever the memory of the moves held before."""
    c = fm.PagedKVCache(12, 4, 2, 64, 2, 4, 20, device=dev)
    c.k.zero_()
    c.v.zero_()
    c.extend(ints([5, 6], dev))
    g = torch.Generator(device=dev).manual_seed(81)
    rows = [rand(g, 11, 2, 64, dtype=torch.bfloat16) for _ in range(2)]
    c.write(*rows)
    path = ints([[0, 2, 4], [0, 1, 5]] + [[0, 1, 2]] * 7, dev)
    slots = c.slots[:11].clone()
    before = [x.clone() for x in (c.k, c.v)]
    for width in (2 * 9 * 3, 2 * 2 * 3):  # slots of the cache in memory that comes back from the allocator
        old = slots.repeat(5)[:width].clone()
        del old
    moves = c.keep(path, ints([3, 3], dev))
    c.move(moves)
    fm.fm_sync_status()
    assert moves.shape == (2, 2, 3) and c.kv_len.tolist() == [3, 3] and c.status.item() == 0
    for x, was in zip((c.k, c.v), before):
        for to, at in ((1, 2), (2, 4), (7, 10)):  # tokens of the step: nodes 2 and 4 of the first row, 5 of the second
            s, d = slots[at].item(), slots[to].item()
            was[d // 4, :, d % 4] = was[s // 4, :, s % 4].clone()
        assert torch.equal(x, was)


@pytest.mark.parametrize("captured", [False, True])
def test_an_extend_that_does_not_fit_is_known_after_the_step(dev, captured):  # noqa: F811
    """extend to move with more drafts than a table's row or the list has pages: nothing changes, and status still says so; the next step
    that fits clears it.  Paths that cannot be are counted apart."""
    g = torch.Generator(device=dev).manual_seed(82)
    c = fm.PagedKVCache(8, 4, 1, 64, 2, 6, 40, device=dev)
    c.k.zero_()
    c.v.zero_()
    new, parent, tokens = ints([0, 0], dev), ints([-1] * 40, dev), ints([0] * 40, dev)
    kept2, use = ints([0, 0], dev), ints([0, 0], dev)
    p, u, last = torch.full((40, 5), 0.2, device=dev), torch.zeros(40, device=dev), torch.zeros(2, device=dev)
    q, k = (rand(g, 40, h, 64, dtype=torch.bfloat16) for h in (2, 1))
    seen = {}

    def step():
        c.extend(new)
        mask = c.tree(parent, 1)
        c.write(k, k)
        c.tree_attention(q, mask)
        path, kept, nxt = fm.verify_tree(p, tokens, parent, c.cu_q, u, last, max_path=4)
        c.move(c.keep(path, torch.where(use != 0, kept2, kept)))
        seen.update(kept=kept, nxt=nxt)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    if captured:
        with torch.cuda.graph(graph):
            step()
    # (u = 0: every first child is kept, four of a chain of drafts)
    for lens, want, ok in (([6, 9], [4, 4], True), ([30, 1], [4, 4], False), ([3, 1], [7, 5], True), ([15, 12], [7, 5], False),
                           ([0, 0], [7, 5], True)):
        new.copy_(ints(lens, dev))
        parent.copy_(ints((list(range(-1, lens[0] - 1)) + list(range(-1, lens[1] - 1)) + [-1] * 40)[:40], dev))
        k0 = c.k.clone()
        graph.replay() if captured else step()
        fm.fm_sync_status()
        assert (c.status.item() == 0) == ok and c.keep_status.item() == 0 and c.kv_len.tolist() == want
        if not ok:
            assert torch.equal(c.k, k0) and seen["kept"].tolist() == [0, 0] and seen["nxt"].tolist() == [-1, -1]
    kept2.copy_(ints([9, 1], dev))
    use.fill_(1)
    new.copy_(ints([2, 1], dev))
    parent.copy_(ints([-1, 0, -1] + [-1] * 37, dev))
    graph.replay() if captured else step()
    fm.fm_sync_status()
    assert c.status.item() == 0 and c.keep_status.item() == 1 and c.kv_len.tolist() == [9, 6]


def expect(case, row_of, first, nodes, at, i, max_path):
    """Path, number and next token of request i by the definition; nothing of a request that is passed over."""
    if first < 0:
        return [-1] * max_path, -1, -1
    target, draft, tokens, parents, u, u_last = case
    sl, r = slice(at, at + nodes), slice(row_of, row_of + nodes)
    p, x = walk(target[r], None if draft is None else draft[r], tokens[sl], parents[sl], u[sl].tolist(), float(u_last[i]), max_path)
    return p + [-1] * (max_path - len(p)), len(p), x


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("dtype,drafted", [(F32, True), (BF16, True), (F16, False)])
def test_verification_passes_over_what_is_no_tree(dev, dtype, drafted, captured):  # noqa: F811
    """Trees whose rows lie in another order than their tokens, chunks of any length among them, of tokens that no
    vocabulary has; rows shared by two requests; captured: replayed with other lengths and rows."""
    g = torch.Generator(device=dev).manual_seed(83)
    V, width, n, T, R = 2003, 7, 6, 3100, 60
    cu, rows, tokens, parent = ints([0] * (n + 1), dev), ints([-1] * n, dev), ints([0] * T, dev), ints([-1] * T, dev)
    target, draft = (torch.zeros(R, V, dtype=dtype, device=dev) for _ in range(2))
    u, last = torch.zeros(T, device=dev), torch.zeros(n, device=dev)
    path, kept, nxt = (Guarded(s, torch.int32, dev) for s in ((n, width), (n,), (n,)))
    call = lambda: fm.fm_tree_verify(target, draft if drafted else None, cu, tokens, parent, u, last, path.t, kept.t, nxt.t,  # noqa: E731
                                     rows=rows)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    if captured:
        with torch.cuda.graph(graph):
            call()
    for new, first in (([9, 1500, 5, 40, 1, 17], [30, -1, 0, -2, 59, 10]), ([20, 20, 0, 0, 1025, 3], [40, 40, 7, -1, -1, 0]),
                       ([1, 2, 3, 4, 5, 6], [-1] * 6), ([0, 1024, 1, 26, 2, 2000], [60, -9, 5, 34, 0, -2 ** 31])):
        at = starts(new)
        c = tree_case(g, [R], V, dtype, drafted)  # rows; the trees' own tokens below
        target.copy_(c[0])
        if drafted:
            draft.copy_(c[1])
        toks, pars = [-5] * T, [7] * T
        for i, (q, f) in enumerate(zip(new, first)):
            if f < 0:
                continue
            tree = random_tree(q, 40 + i, 4)
            pars[at[i]:at[i] + q] = tree
            for t in range(1, q):
                row = (c[1] if drafted else c[0])[f + tree[t]].float()
                toks[at[i] + t] = int(torch.multinomial(row, 1, generator=g))
        tokens.copy_(ints(toks, dev))
        parent.copy_(ints(pars, dev))
        u.copy_(torch.rand(T, generator=g, device=dev) * 0.6)
        last.copy_(torch.rand(n, generator=g, device=dev))
        cu.copy_(ints(at, dev))
        rows.copy_(ints(first, dev))
        for x in (path, kept, nxt):
            x.t.fill_(-7)
        graph.replay() if captured else call()
        fm.fm_sync_status()
        case = (c[0], c[1], toks, pars, u, last)
        for i in range(n):
            want = expect(case, first[i], first[i], new[i], at[i], i, width)
            assert (path.t[i].tolist(), kept.t[i].item(), nxt.t[i].item()) == want, i
        assert all(x.intact() for x in (path, kept, nxt))


def test_rows_that_the_target_does_not_have_are_reported(dev):  # noqa: F811
    p, f = torch.full((10, 16), 1 / 16, device=dev), lambda n: torch.zeros(n, device=dev)  # noqa: E731
    for first, count in ((8, 3), (10, 1), (2 ** 31 - 1, 3), (0, 1025)):
        call = lambda r: fm.verify_tree(p, ints([1] * 1030, dev), ints([-1] + list(range(1029)), dev), ints([0, count, count + 2], dev),  # noqa: E731
                                        f(1030), f(2), max_path=4, rows=ints(r, dev))
        path, kept, nxt = call([first, 8])
        with pytest.raises(fm.FMError, match="request 0 do not fit") as e:
            fm.fm_sync_status()
        assert e.value.code == fm.FM_ERR_INDEX and kept.tolist()[0] == 0 and nxt.tolist()[0] == -1 and (path[0] == -1).all()
        call([-1, 8])
        fm.fm_sync_status()
    # no rows at all, and nobody who wants one
    path, kept, nxt = fm.verify_tree(p[:0], ints([0] * 5, dev), ints([-1] * 5, dev), ints([0, 5, 5], dev), f(5), f(2), rows=ints([-1, 0], dev))
    fm.fm_sync_status()
    assert kept.tolist() == [-1, 0] and nxt.tolist() == [-1, -1] and (path == -1).all()


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("drafted", [True, False])
def test_prompt_chunks_beside_trees_from_extend_to_move(dev, drafted, captured):  # noqa: F811
    """A chunk of more tokens than a mask row has bits and a short one, which is a chain, beside two trees: nothing is
    reported, chunks keep all they have, trees what the definition keeps."""
    g, r = torch.Generator(device=dev).manual_seed(84), random.Random(85)
    n, ps, Hq, Hk, D, V, width, cap, R = 4, 16, 4, 2, 64, 300, 6, 1700, 40
    c = fm.PagedKVCache(600, ps, Hk, D, n, 300, cap, device=dev)
    c.k.fill_(float("nan"))
    c.v.fill_(float("nan"))
    new_d, parent, tokens, first = ints([0] * n, dev), ints([-1] * cap, dev), ints([0] * cap, dev), ints([-1] * n, dev)
    q, k, v = (torch.zeros(cap, h, D, dtype=BF16, device=dev) for h in (Hq, Hk, Hk))
    out, lse = torch.zeros(cap, Hq, D, dtype=BF16, device=dev), torch.zeros(Hq, cap, device=dev)
    target, draft = (torch.zeros(R, V, device=dev) for _ in range(2))
    u, last = torch.zeros(cap, device=dev), torch.zeros(n, device=dev)
    seen = {}

    def step():
        c.extend(new_d)
        mask = c.tree(parent)  # (1,024 bits: the longer chunks are causal)
        c.write(k, v)
        c.tree_attention(q, mask, out=out, lse=lse)
        path, kept, nxt = fm.verify_tree(target, tokens, parent, c.cu_q, u, last, draft if drafted else None, width, rows=first)
        c.move(c.keep(path, kept))
        seen.update(path=path, kept=kept, nxt=nxt)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    if captured:
        with torch.cuda.graph(graph):
            step()
    hist = [tuple(torch.zeros(0, Hk, D) for _ in range(2)) for _ in range(n)]
    moved = 0
    for new, chunk in (([300, 40, 1100, 7], (1, 1, 1, 1)), ([9, 1500, 12, 40], (0, 1, 0, 1)), ([17, 5, 1200, 11], (0, 0, 1, 0))):
        at, T = starts(new), sum(new)
        trees = [list(range(-1, a - 1)) if x else random_tree(a, r.randrange(999), 4) for a, x in zip(new, chunk)]
        row_of, rows_used = [-1] * n, 0
        for i in reversed(range(n)):
            if not chunk[i]:
                row_of[i], rows_used = rows_used, rows_used + new[i]
        target.copy_(torch.softmax(torch.randn(R, V, generator=g, device=dev) * 2, 1))
        draft.copy_(torch.softmax(torch.log(target) + 0.4 * torch.randn(R, V, generator=g, device=dev), 1))
        toks = [V + 5] * cap
        for i in range(n):
            for t in range(new[i] if not chunk[i] else 0):
                toks[at[i] + t] = int(torch.multinomial(draft[row_of[i] + max(trees[i][t], 0)], 1, generator=g))
        tokens.copy_(ints(toks, dev))
        parent[:T] = ints(sum(trees, []), dev)
        for x in (q, k, v):
            x.copy_(rand(g, *x.shape, dtype=BF16))
        u.copy_(torch.rand(cap, generator=g, device=dev) * (1.0 if drafted else 0.1))
        last.copy_(torch.rand(n, generator=g, device=dev))
        new_d.copy_(ints(new, dev))
        first.copy_(ints(row_of, dev))
        graph.replay() if captured else step()
        fm.fm_sync_status()
        assert c.status.item() == 0 and c.keep_status.item() == 0
        case = (target, draft if drafted else None, toks, sum(trees, []), u, last)
        for i in range(n):
            a, sl, was = new[i], slice(at[i], at[i + 1]), hist[i][0].shape[0]
            want = expect(case, row_of[i], row_of[i], a, at[i], i, width)
            assert (seen["path"][i].tolist(), seen["kept"][i].item(), seen["nxt"][i].item()) == want, i
            stay = list(range(a)) if chunk[i] else want[0][:want[1]]
            moved += sum(j != x for j, x in enumerate(stay))
            K, W = (torch.cat([h, x[sl].float().cpu()]) for h, x in zip(hist[i], (k, v)))
            see = causal_seen(a, was + a) if chunk[i] else tree_seen(mask_words(trees[i], 2), was + a)
            assert_close(out[sl], lse[:, sl], *attend_seen(q[sl], K, W, see, D ** -0.5), BF16, BF16, D, was + a)
            hist[i] = tuple(torch.cat([h, x[sl].float().cpu()[stay]]) for h, x in zip(hist[i], (k, v)))
        assert c.kv_len.tolist() == [h[0].shape[0] for h in hist]
        for i in range(n):  # the cache holds each history
            slot = torch.arange(hist[i][0].shape[0], device=dev)
            page = c.block_table[i].long()[slot // ps]
            for x, h in zip((c.k, c.v), hist[i]):
                assert torch.equal(x[page, :, slot % ps].float().cpu(), h)
    assert moved > 0
