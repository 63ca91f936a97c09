"""Plain 64-bit reference of attention over requests of different lengths, and the error bound of
a kernel that rounds where the package says it does."""
import math

import torch

HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def attend(q, k, v, causal, window, scale):
    """One request: q [t, Hq, D], k, v [s, Hk, D] -> o [t, Hq, D], lse [Hq, t], the mean |v| that each
    output weighs, and the largest sum of |q_d k_d| * scale, in float64 on the CPU."""
    t, Hq, D = q.shape
    s, Hk = k.shape[0], k.shape[1]
    q, k, v = q.double().cpu(), k.double().cpu(), v.double().cpu()
    o, a = torch.zeros(t, Hq, D, dtype=torch.float64), torch.zeros(t, Hq, D, dtype=torch.float64)
    lse = torch.full((Hq, t), -math.inf, dtype=torch.float64)
    big = 0.0
    pos = torch.arange(t)[:, None] + (s - t)
    j = torch.arange(s)[None]
    seen = torch.ones(t, s, dtype=torch.bool) if not causal else (j <= pos) & ((j > pos - window) if window else True)
    rows = seen.any(1)
    if s == 0 or not rows.any():
        return o, lse, a, big
    for h in range(Hq):
        kh, vh = k[:, h // (Hq // Hk)], v[:, h // (Hq // Hk)]
        x = (q[:, h] @ kh.T) * scale
        big = max(big, float((q[:, h].abs() @ kh.abs().T).max()) * scale)
        x = x.masked_fill(~seen, -math.inf)
        p = torch.softmax(x[rows], 1)
        o[rows, h] = p @ vh
        a[rows, h] = p @ vh.abs()
        lse[h, rows] = torch.logsumexp(x[rows], 1)
    return o, lse, a, big


def check(o, lse, ref_o, ref_lse, ref_a, big, in_dtype, D, keys):
    """|o - ref| within: half a step of the input type for each weight p (16-bit inputs: p is
    rounded to it before it meets v) and half a step of o's type, and fp32 arithmetic: each score's
    dot product of D terms is off by at most (D + 2) 2^-24 sum |q_d k_d|, which moves p by that
    relative amount in the numerator and in the denominator, and sums of n terms by n 2^-24."""
    o, lse = o.double().cpu(), None if lse is None else lse.double().cpu()
    eps32 = 2.0 ** -24
    score = (D + 4) * eps32 * big
    arith = 2 * score + 2 * (keys + 8) * eps32
    up = 0.0 if in_dtype == torch.float32 else HALF_STEP[in_dtype]
    return o, lse, score, arith, up


def assert_close(o, lse, ref_o, ref_lse, ref_a, big, in_dtype, out_dtype, D, keys):
    o, lse, score, arith, up = check(o, lse, ref_o, ref_lse, ref_a, big, in_dtype, D, keys)
    bound = (up + arith) * 1.01 * ref_a + HALF_STEP[out_dtype] * 1.01 * ref_o.abs()
    if out_dtype == torch.float16:
        bound = bound + 2.0 ** -25  # half a step of fp16's subnormals
    err = (o - ref_o).abs()
    assert torch.isfinite(o).all()
    bad = err > bound
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} outputs out of bound, worst by "
                           f"{float((err - bound).max()):.3g} at {torch.nonzero(bad)[0].tolist()}")
    if lse is not None:
        empty = torch.isinf(ref_lse)
        assert torch.equal(torch.isneginf(lse), empty)
        # the sum's relative error, and one rounding of max + log2(sum) and of its factor ln 2
        lb = score + (keys + 8) * eps(ref_lse[~empty])
        assert ((lse - ref_lse).abs()[~empty] <= lb).all(), float((lse - ref_lse).abs()[~empty].max())


def eps(x):
    return 2.0 ** -24 * (1.0 + x.abs())
