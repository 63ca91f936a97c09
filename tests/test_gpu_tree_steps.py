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
