"""Out-of-bounds write checks of the calls over requests of different lengths: every buffer that they
write (outputs, LSE, a workspace of exactly the stated size, caches, tables, lists, slot maps)
lies between guard bands that hold a fixed pattern and must still hold it afterwards."""
import pytest
import torch

import fixed_max_softmax_gb300 as fm
from tests.test_gpu_guard_bands import GUARD, PATTERN, Guarded
from tests.test_gpu_seqs import BF16, DECODE, F16, F32, MIXED, check_paged, check_varlen, dev, ints, paged_case, rand, starts  # noqa: F401

pytestmark = pytest.mark.gpu
PATTERN.setdefault(F16, (torch.int16, 0x7E01))


class Space:
    """A workspace of exactly nbytes between two bands of 4 KiB."""

    def __init__(self, nbytes, dev):
        self.flat = torch.full((nbytes + 2 * GUARD,), 0xA5, dtype=torch.uint8, device=dev)
        self.t, self.n = self.flat[GUARD:GUARD + nbytes], nbytes

    def intact(self):
        return bool((self.flat[:GUARD] == 0xA5).all()) and bool((self.flat[GUARD + self.n:] == 0xA5).all())


LONG = [(1, 9000), (300, 4000), (2, 40)]
PROMPTS = [(700, 700), (1, 1), (129, 129), (64, 64)]


@pytest.mark.parametrize("lens", [DECODE, MIXED, LONG, [(1, 20000)], [(1, 3)] * 500])
@pytest.mark.parametrize("dtype,out,D,Hq,Hk,ps", [(BF16, BF16, 128, 10, 2, 16), (F16, F32, 64, 7, 1, 128), (F32, F32, 128, 4, 2, 16),
                                                 (BF16, F32, 128, 6, 6, 5)])
def test_paged_stays_inside(dev, dtype, out, D, Hq, Hk, ps, lens):  # noqa: F811
    g = torch.Generator(device=dev).manual_seed(30)
    ks, vs, kc, vc, table = paged_case(g, lens, Hk, D, ps, dtype, True)
    T = sum(a for a, _ in lens)
    q = rand(g, T, Hq, D, dtype=dtype)
    o, lse = Guarded((T, Hq, D), out, dev, pad=32), Guarded((Hq, T), F32, dev)
    ws = Space(fm.fm_attn_seqs_workspace_size(len(lens), T, Hq, Hk, D), dev)
    fm.fm_attn_paged(q, kc, vc, ints(starts([a for a, _ in lens]), dev), ints([b for _, b in lens], dev), table, fm.seqs_opts(),
                     o.t, lse.t, ws.t)
    fm.fm_sync_status()
    assert o.intact() and lse.intact() and ws.intact()
    n = min(len(lens), 8)
    rows = sum(a for a, _ in lens[:n])
    check_paged(q[:rows], ks, vs, lens[:n], o.t[:rows], lse.t[:, :rows])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens", [PROMPTS, LONG, [(1, 1)]])
def test_varlen_stays_inside(dev, dtype, lens):  # noqa: F811
    g = torch.Generator(device=dev).manual_seed(31)
    T, Tk = sum(a for a, _ in lens), sum(b for _, b in lens)
    q, k, v = (rand(g, n, h, 128, dtype=dtype) for n, h in ((T, 5), (Tk, 1), (Tk, 1)))
    o, lse = Guarded((T, 5, 128), dtype, dev, pad=8), Guarded((5, T), F32, dev)
    ws = Space(fm.fm_attn_seqs_workspace_size(len(lens), T, 5, 1, 128), dev)
    fm.fm_attn_varlen(q, k, v, ints(starts([a for a, _ in lens]), dev), ints(starts([b for _, b in lens]), dev), fm.seqs_opts(),
                      o.t, lse.t, ws.t)
    fm.fm_sync_status()
    assert o.intact() and lse.intact() and ws.intact()
    check_varlen(q, k, v, lens, o.t, lse.t, True, 0)


@pytest.mark.parametrize("n,cap,ps", [(1, 1, 16), (7, 40, 4), (1025, 3001, 16), (30, 9999, 8)])
def test_extend_and_write_stay_inside(dev, n, cap, ps):  # noqa: F811
    width, pages = 9, n * 4 + 8
    table, free = Guarded((n, width), torch.int32, dev, pad=3), Guarded((pages,), torch.int32, dev)
    kv, cu, status = Guarded((n,), torch.int32, dev), Guarded((n + 1,), torch.int32, dev), Guarded((1,), torch.int32, dev)
    count, slots, pos = Guarded((1,), torch.int32, dev), Guarded((2 * cap,), torch.int32, dev), Guarded((cap,), torch.int32, dev)
    slots64 = slots.t.view(torch.int64)
    every = (table, free, kv, cu, status, count, slots, pos)
    free.t.copy_(torch.arange(pages - 1, -1, -1))
    count.t.fill_(pages)
    kv.t.zero_()
    table.t.fill_(-1)
    kc, vc = (Guarded((pages, 2, ps, 64), BF16, dev) for _ in range(2))
    rows = torch.ones(cap, 2, 64, dtype=BF16, device=dev)
    release = torch.zeros(n, dtype=torch.uint8, device=dev)
    release[::3] = 1
    for step, new in enumerate((min(cap // n, ps + 1), 1 if cap >= n else 0, 10 ** 6, 2 * ps if 2 * ps * n <= cap else 0)):
        fm.fm_paged_extend(ints([new] * n, dev), release if step == 3 else None, kv.t, kv.t, table.t, free.t, count.t, count.t, ps,
                           cu.t, slots64, pos.t, status.t)
        fm.fm_paged_write(rows, rows, slots64, kc.t, vc.t)
        fm.fm_sync_status()
        assert all(b.intact() for b in every) and kc.intact() and vc.intact(), step
        assert (status.t.item() == 0) == (new < 10 ** 6)


@pytest.mark.parametrize("shift", [16, 32, 48, 112])
@pytest.mark.parametrize("dtype,D,ps", [(BF16, 128, 16), (F16, 64, 128), (F32, 64, 16), (BF16, 128, 5)])
@pytest.mark.parametrize("lens", [LONG, [(1, 9000)], [(400, 5000)]])
def test_workspace_at_any_16_byte_boundary(dev, shift, dtype, D, ps, lens):  # noqa: F811
    """Units cut along their keys, so that partial results are stored: in a workspace of exactly the stated size
    that begins 16, 32, 48 or 112 bytes past a 128-byte line, as one cut from a pool may."""
    g = torch.Generator(device=dev).manual_seed(32)
    ks, vs, kc, vc, table = paged_case(g, lens, 2, D, ps, dtype, True)
    T = sum(a for a, _ in lens)
    q = rand(g, T, 10, D, dtype=dtype)
    o, lse = torch.full_like(q, 7.0), torch.full((10, T), 7.0, device=dev)
    nbytes = fm.fm_attn_seqs_workspace_size(len(lens), T, 10, 2, D)
    whole = Space(nbytes + shift, dev)
    ws = whole.t[shift:]
    assert ws.data_ptr() % 128 == shift and ws.numel() == nbytes
    fm.fm_attn_paged(q, kc, vc, ints(starts([a for a, _ in lens]), dev), ints([b for _, b in lens], dev), table, fm.seqs_opts(),
                     o, lse, ws)
    fm.fm_sync_status()
    assert whole.intact() and bool((whole.t[:shift] == 0xA5).all())
    check_paged(q, ks, vs, lens, o, lse)
