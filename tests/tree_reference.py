"""Plain 64-bit references of the calls on trees of drafted tokens."""
import math
import random

import torch


def random_tree(nodes, seed, back=8):
    """Parents of a tree: node 0 the root, each other node's parent among the `back` nodes before it."""
    r = random.Random(seed)
    return ([-1] + [r.randrange(max(0, t - back), t) for t in range(1, nodes)])[:nodes]


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


def _some(row):
    row = row.double().cpu()
    return torch.where((row > 0) & (row < math.inf), row, torch.zeros_like(row))


def walk(target, draft, tokens, parent, u, u_last, max_path):
    """One request by the definition, in 64 bits: target, draft [nodes, V] (draft may be None); (path, next token).  The
    refusals follow one another, each from what the last one left."""
    V = target.shape[1]
    one = lambda x: 0.0 if math.isnan(x) else min(max(x, 0.0), 1.0)  # noqa: E731
    if len(tokens) == 0:
        return [], -1
    path = [0]
    while True:
        at, grown = path[-1], False
        p = _some(target[at])
        q = _some(draft[at]) if draft is not None else None
        left, mass = p.clone(), 1.0
        for t in range(at + 1, len(tokens)):
            if parent[t] != at or not 0 <= tokens[t] < V or len(path) >= max_path:
                continue
            x = tokens[t]
            if one(u[t]) * (1.0 if q is None else float(q[x])) * mass < float(left[x]):
                path.append(t)
                grown = True
                break
            if q is None:
                mass = max(mass - float(left[x]), 0.0)
                left[x] = 0.0
            else:
                left = (left - mass * q).clamp(min=0)
                mass = float(left.sum())
                if not mass > 0:
                    left, mass = p.clone(), 1.0
        if not grown:
            break
    if not float(left.sum()) > 0:
        left = p
    have = torch.nonzero(left).flatten()
    if len(have) == 0:
        return path, -1
    upto = left.cumsum(0)
    return path, min(int((upto <= one(u_last) * float(upto[-1])).sum()), int(have[-1]))
