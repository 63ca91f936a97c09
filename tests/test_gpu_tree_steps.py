"""Steps with drafted tokens through PagedKVCache and verify_tree() as a program makes them, where parts of a step go
wrong or are not trees."""
import pytest
import torch

import fixed_max_softmax_gb300 as fm
from tests.test_gpu_seqs import dev, ints, rand  # noqa: F401

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
