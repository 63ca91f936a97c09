"""Plain 64-bit references of the calls on trees of drafted tokens."""
import math
import random

import torch


def random_tree(nodes, seed, back=8):
    """Parents of a tree: node 0 the root, each other node's parent among the `back` nodes before it."""
    r = random.Random(seed)
    return [-1] + [r.randrange(max(0, t - back), t) for t in range(1, nodes)]


def ancestors(parent):
    """For each node the set of itself and its ancestors."""
    seen = []
    for t, p in enumerate(parent):
        seen.append((seen[p] if p >= 0 else set()) | {t})
    return seen


def mask_words(parent, words):
    """Rows of 32-bit words, as signed integers."""
    rows = []
    for s in ancestors(parent):
        w = [sum(1 << (j % 32) for j in s if j // 32 == i) for i in range(words)]
        rows.append([x - (1 << 32) if x >= 1 << 31 else x for x in w])
    return rows


def tree_seen(rows, kv):
    """[t, s] which of its request's kv keys each new token sees, from mask rows (bits of later tokens are not looked
    at); rows None: causal."""
    t, words = (len(rows), len(rows[0])) if rows else (0, 0)
    seen = torch.zeros(t, kv, dtype=torch.bool)
    for x in range(t):
        for j in range(kv):
            n = j - (kv - t)
            seen[x, j] = n < 0 or (n <= x and n // 32 < words and bool((rows[x][n // 32] >> (n % 32)) & 1))
    return seen


def causal_seen(t, kv):
    return torch.arange(kv)[None] <= torch.arange(t)[:, None] + (kv - t)


def attend_seen(q, k, v, seen, scale):
    """One request: q [t, Hq, D], k, v [s, Hk, D], seen [t, s] -> o, lse, the mean |v| that each output weighs and the
    largest sum of |q_d k_d| * scale, in float64 on the CPU."""
    t, Hq, D = q.shape
    s, Hk = k.shape[0], k.shape[1]
    q, k, v = q.double().cpu(), k.double().cpu(), v.double().cpu()
    o, a = torch.zeros(t, Hq, D, dtype=torch.float64), torch.zeros(t, Hq, D, dtype=torch.float64)
    lse = torch.full((Hq, t), -math.inf, dtype=torch.float64)
    big, rows = 0.0, seen.any(1)
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
