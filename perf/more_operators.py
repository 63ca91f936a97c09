"""Serving with drafted tokens over the paged cache as measured workloads.

Each request brings a tree of tokens drafted for it: node 0 is the last token that is certain, a node's
children are guesses at the token after it.

    mask    fm_tree_mask: which nodes each node sees (itself and its ancestors) and its position
    tree    fm_attn_tree: attention of the nodes over their request's pages and, in the tree, over their
            ancestors; prompt chunks in the same call are causal
    verify  fm_tree_verify: the walk down each tree that keeps a node or not by the target's
            probabilities and given random numbers, and the token after the last node kept
    keep    fm_paged_write, fm_paged_keep, fm_paged_move: the nodes' rows put into the cache, then the
            cache cut back to the nodes that are kept: lengths, pages, rows
    step    all of them in a row, as one layer of a step with drafts

`run` computes them in plain torch operations, or with `own` true through the package's entry points.
Lengths, trees and kept paths are a function of the case alone (its `mix` seeds them), values of the seed; where a
call's values are the trees themselves, so are they.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


def _case(name, kind, **kw):
    c = {"kind": kind, "dtype": "bf16", "n": 1, "nodes": 26, "ragged": False, "chain": False, "chunks": 0, "q_max": 1,
         "kv_max": 1024, "heads": 32, "kv_heads": 8, "head_dim": 128, "page": 16, "token_major": True, "vocab": 32000,
         "drafted": True, "mix": 1}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one user's draft tree, before a step: latency alone
        _case("mask one 26", "mask", n=1, kv_max=900, mix=1),
        # a full batch of large trees of different sizes
        _case("mask batch 256", "mask", n=256, nodes=64, ragged=True, kv_max=4000, mix=2),
        # one user's tree over a short context
        _case("tree one 900", "tree", n=1, kv_max=900, mix=3),
        # a batch of small trees, contexts of all lengths, 5 query heads to a key head
        _case("tree batch 32", "tree", n=32, nodes=16, ragged=True, kv_max=8192, heads=40, mix=4),
        # few users with long contexts and large trees, one page's head rows together
        _case("tree long 65k fp16", "tree", n=4, nodes=64, kv_max=65536, heads=64, page=64, dtype="fp16",
              token_major=False, mix=5),
        # a handful of small trees in full precision
        _case("tree small fp32", "tree", n=5, nodes=9, ragged=True, kv_max=700, heads=12, kv_heads=12, head_dim=64,
              dtype="fp32", mix=7),
        # one user's tree, children sampled from the draft model
        _case("verify one 32k", "verify", n=1, nodes=9, dtype="fp32", mix=8),
        # a batch of chains of 5 sampled tokens over a large vocabulary
        _case("verify chains 64", "verify", n=64, nodes=6, chain=True, vocab=128000, dtype="fp32", mix=9),
        # a batch of trees of chosen (not sampled) tokens, an odd vocabulary, 16-bit probabilities
        _case("verify trees 48", "verify", n=48, ragged=True, vocab=100003, drafted=False, mix=10),
        # one user's nodes, the way down of a few kept
        _case("keep one 26", "keep", n=1, kv_max=900, mix=13),
        # a batch's nodes written, the kept ones moved together; two prompt chunks keep all they have
        _case("keep 64", "keep", n=64, nodes=26, ragged=True, chunks=2, q_max=300, kv_max=4000, mix=11),
        # one layer of a whole step with drafts
        _case("step 32", "step", n=32, nodes=21, ragged=True, kv_max=4096, heads=40, mix=12),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["mask", "tree", "tree", "tree", "tree", "verify", "verify", "verify", "keep", "step"])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 10])
    group = rng.choice([1, 2, 4, 4, 5, 7, 8])
    c = _case(None, kind, mix=rng.randrange(1 << 20), kv_heads=kv_heads, heads=kv_heads * group, ragged=rng.random() < 0.7,
              chain=rng.random() < 0.2, head_dim=rng.choice([64, 128, 128]),
              dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), page=rng.choice([8, 16, 16, 32, 64, 128]),
              token_major=rng.random() < 0.5, nodes=_between(rng, 2, 70), drafted=rng.random() < 0.6)
    if kind == "mask":
        c.update(n=_between(rng, 1, 256), kv_max=_between(rng, 100, 9000), nodes=max(10, c["nodes"]), chain=False)
        return c
    if kind in ("verify", "step"):
        c.update(vocab=_between(rng, 500, 130000 if kind == "verify" else 32000), n=_between(rng, 1, 64), kv_max=_between(rng, 100, 4000))
        while c["n"] * c["nodes"] * c["vocab"] > (100000000 if kind == "verify" else 20000000):
            c["n"], c["nodes"] = (c["n"] + 1) // 2, max(2, c["nodes"] * 3 // 4)
    else:
        c.update(n=_between(rng, 1, 64), kv_max=_between(rng, 100, 32000 if kind == "tree" else 6000))
        while c["n"] * c["kv_max"] > 200000:
            c["n"] = (c["n"] + 1) // 2
        if rng.random() < 0.3 and c["n"] > 1:
            c.update(chunks=rng.randint(1, min(3, c["n"] - 1)), q_max=_between(rng, 100, 500))
    if c["dtype"] == "fp32" and kind in ("tree", "step"):
        c.update(n=min(c["n"], 8), kv_max=min(c["kv_max"], 2000), nodes=min(c["nodes"], 24), chunks=0)
    return c


def _words(c):
    return -(-c["nodes"] // 32)


def _requests(c, seed=None):
    """(new tokens, keys with the new ones, parents or None, kept path or None) of each request; the first has the
    case's largest.  The last `chunks` requests bring a prompt chunk, of more tokens than the mask has bits.  With a
    seed the trees are the seed's, else the case's."""
    rng, shape = random.Random(c["mix"]), random.Random(c["mix"] if seed is None else seed)
    out = []
    for i in range(c["n"]):
        s = c["kv_max"] if i == 0 else _between(rng, max(1, c["kv_max"] // 16), c["kv_max"])
        if i >= c["n"] - c["chunks"]:
            q = max(32 * _words(c) + 1, _between(rng, max(1, c["q_max"] // 4), c["q_max"]))
            out.append((q, max(q, s), None, None))
            continue
        q = c["nodes"] if i == 0 or not c["ragged"] else _between(rng, max(1, c["nodes"] // 3), c["nodes"])
        parent = [-1] + [t - 1 if c["chain"] else shape.randrange(max(0, t - 8), t) for t in range(1, q)]
        path = [0]
        for t in range(1, q):
            if parent[t] == path[-1] and shape.random() < 0.6:
                path.append(t)
        out.append((q, max(q, s), parent, path))
    return out


def _ancestors(parent):
    """For each node its ancestors and itself."""
    seen = []
    for t, p in enumerate(parent):
        seen.append((seen[p] if p >= 0 else []) + [t])
    return seen


def _longest(reqs):
    """Nodes on the longest way down a tree."""
    return max([1] + [max(map(len, _ancestors(p))) for _, _, p, _ in reqs if p])


def work(case):
    c, es = case, BYTES[case["dtype"]]
    reqs = _requests(c)
    n, t = c["n"], sum(q for q, _, _, _ in reqs)
    row = c["kv_heads"] * c["head_dim"] * es
    total = {"bytes": 0, "flops": 0}

    def add(bytes_, flops=0.0):
        total["bytes"] += bytes_
        total["flops"] += flops

    if c["kind"] in ("mask", "step"):  # parents; a mask row and a position for each node
        add(4 * t + 8 * n + 4 * t * _words(c) + 4 * t)
    if c["kind"] in ("tree", "step"):
        pairs = keys = 0
        for q, s, parent, _ in reqs:
            keys += s
            pairs += q * (s - q) + (sum(map(len, _ancestors(parent))) if parent else q * (q + 1) // 2)
        add(2 * t * c["heads"] * c["head_dim"] * es + 4 * t * c["heads"] + 2 * keys * row + 8 * n + 4 * t * _words(c)
            + 4 * sum(-(-s // c["page"]) for _, s, _, _ in reqs), 4.0 * pairs * c["heads"] * c["head_dim"])
    if c["kind"] in ("verify", "step"):  # one row of the target for each request, and of the draft
        rows = n * (2 if c["drafted"] else 1)
        add(rows * c["vocab"] * es + 12 * t + 12 * n + 4 * n * _longest(reqs), 2.0 * rows * c["vocab"])
    if c["kind"] in ("keep", "step"):  # rows written; rows of kept nodes that are not in their place read and written
        moved = sum(sum(x != j for j, x in enumerate(path)) for _, _, _, path in reqs if path)
        add(4 * t * row + 8 * t + 4 * moved * row + n * (16 + 20 * _longest(reqs)))
    return total


def _cache_of(c, pages, make):
    shape = (pages, c["page"], c["kv_heads"], c["head_dim"]) if c["token_major"] else (
        pages, c["kv_heads"], c["page"], c["head_dim"])
    t = make(shape)
    return t.transpose(1, 2) if c["token_major"] else t  # [pages, kv heads, page, head dim] either way


def _probabilities(c, s, g):
    """Distributions of the target and of the draft model after each node, and the nodes' tokens: some tokens of each
    row stand out, and the draft sees them with some noise."""
    dev, dt, v, t = "cuda", DTYPES[c["dtype"]], c["vocab"], s["tokens_total"]
    rand = lambda *shape: torch.randn(shape, generator=g, device=dev)  # noqa: E731
    logits = rand(t, v) * 1.5
    stand_out = torch.randint(0, v, (t, 6), generator=g, device=dev)
    logits.scatter_add_(1, stand_out, rand(t, 6) * 2 + math.log(v))
    s["target"] = torch.softmax(logits, 1).to(dt)
    logits += rand(t, v) * 0.5
    draft = torch.softmax(logits, 1).to(dt)
    most = max([1] + [max(p.count(x) for x in p) for _, _, p, _ in s["reqs"] if p and len(p) > 1])
    if c["drafted"]:
        s["draft"] = draft
        cdf = draft.float().cumsum(1)
        guesses = torch.searchsorted(cdf, torch.rand((t, most), generator=g, device=dev) * cdf[:, -1:]).clamp(max=v - 1)
    else:
        s["draft"] = None
        guesses = draft.float().topk(min(most, v), 1).indices
    at, rows, cols = 0, [], []
    for q, _, parent, _ in s["reqs"]:
        count = [0] * q
        for x in range(q):
            p = max(0, parent[x])
            rows.append(at + p)
            cols.append(count[p])
            count[p] += x > 0
        at += q
    s["node_tokens"] = guesses[torch.tensor(rows, device=dev), torch.tensor(cols, device=dev)].to(torch.int32)
    s["u"] = torch.rand(t, generator=g, device=dev)
    s["u_last"] = torch.rand(c["n"], generator=g, device=dev)


def prepare(case, seed):
    c, dt, dev = case, DTYPES[case["dtype"]], "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    rand = lambda *shape: torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dt)  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    reqs = _requests(c, seed if c["kind"] == "mask" else None)
    new, total = [r[0] for r in reqs], [r[1] for r in reqs]
    n, t, width = c["n"], sum(new), _longest(reqs)
    cu = [0]
    for q in new:
        cu.append(cu[-1] + q)
    parents = []
    for q, _, p, _ in reqs:
        parents += p if p else range(-1, q - 1)
    s = {"case": c, "reqs": reqs, "new": new, "total": total, "tokens_total": t, "cu": cu, "cu_q": ints(cu), "kv_len": ints(total),
         "parent": ints(parents), "width": width, "depth": width}
    if c["kind"] in ("mask", "step"):
        s["mask_out"] = torch.zeros((t, _words(c)), dtype=torch.int32, device=dev)
        s["positions"] = torch.zeros(t, dtype=torch.int32, device=dev)
    if c["kind"] == "mask":
        return s
    if c["kind"] in ("verify", "step"):
        _probabilities(c, s, g)
        s["path"] = torch.zeros((n, width), dtype=torch.int32, device=dev)
        s["kept"], s["next"] = ints([0] * n), ints([0] * n)
    if c["kind"] == "verify":
        return s
    if c["kind"] in ("tree", "step"):
        sharp = torch.rand((c["heads"], 1), generator=g, device=dev) * 1.5 + 0.5  # heads look with different sharpness
        s["q"] = (torch.randn((t, c["heads"], c["head_dim"]), generator=g, device=dev) * sharp).to(dt)
        s["o"] = torch.empty((t, c["heads"], c["head_dim"]), dtype=dt, device=dev)
        s["lse"] = torch.empty((c["heads"], t), dtype=torch.float32, device=dev)
    # a cache with every page that the requests need and some more, its pages dealt out in random order
    ps = c["page"]
    need = [-(-x // ps) for x in total]
    pages = sum(need) + sum(need) // 8 + 16
    order = torch.randperm(pages, generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    s["table"] = torch.full((n, max(need) + 1), -1, dtype=torch.int32, device=dev)
    req = torch.repeat_interleave(torch.arange(n, device=dev), torch.tensor(need, device=dev))
    start = torch.tensor([sum(need[:i]) for i in range(n)], device=dev)
    s["table"][req, torch.arange(sum(need), device=dev) - start[req]] = order[: sum(need)]
    s["k_cache"] = _cache_of(c, pages, lambda shape: rand(*shape))
    s["v_cache"] = _cache_of(c, pages, lambda shape: rand(*shape))
    if c["kind"] == "tree":  # the nodes' masks, in hand since the step began
        s["mask"] = _pack(_dense_mask(s), _words(c))
        return s
    # the new tokens' rows and slots; the list of free pages
    s["k"], s["v"] = rand(t, c["kv_heads"], c["head_dim"]), rand(t, c["kv_heads"], c["head_dim"])
    req = torch.repeat_interleave(torch.arange(n, device=dev), torch.tensor(new, device=dev))
    pos = torch.arange(t, device=dev) - s["cu_q"][req] + (torch.tensor(total, device=dev) - torch.tensor(new, device=dev))[req]
    s["slots"] = s["table"][req, pos // ps].long() * ps + pos % ps
    free = pages - sum(need)
    s["free"] = torch.full((pages,), -1, dtype=torch.int32, device=dev)
    s["free"][:free] = order[sum(need):]
    s["count"], s["count_out"], s["kv_out"], s["status"] = ints([free]), ints([0]), ints([0] * n), ints([0])
    s["src"] = torch.zeros((n, width), dtype=torch.int64, device=dev)
    s["dst"] = torch.zeros((n, width), dtype=torch.int64, device=dev)
    if c["kind"] == "keep":
        s["path"] = ints([(p or []) + [-1] * (width - len(p or [])) for _, _, _, p in reqs])
        s["kept"] = ints([len(p) if p else -1 for _, _, _, p in reqs])
    return s


# ---------------------------------------------------------------- plain forms
def _dense_mask(s):
    """[T, nodes]: node t of a tree sees node j of its request (prompt chunks: nothing set)."""
    c, dev = s["case"], s["cu_q"].device
    t, first = s["tokens_total"], s["cu_q"][:-1].long()
    req = torch.repeat_interleave(torch.arange(c["n"], device=dev), (s["cu_q"][1:] - s["cu_q"][:-1]).long(), output_size=t)
    at = torch.arange(t, device=dev)
    tree = (s["cu_q"][1:] - s["cu_q"][:-1])[req] <= 32 * _words(c)
    seen = torch.zeros((t, 32 * _words(c)), dtype=torch.bool, device=dev)
    here = torch.where(tree, at - first[req], -1)
    for _ in range(s["depth"]):
        on = here >= 0
        j = here.clamp(min=0)
        seen.scatter_(1, j[:, None], (seen.gather(1, j[:, None]) | on[:, None]))
        here = torch.where(on, s["parent"][first[req] + j].long(), -1)
    return seen


def _pack(seen, words):
    bit = torch.arange(32, device=seen.device)
    w = (seen.view(seen.shape[0], words, 32).long() << bit).sum(2)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def _unpack(mask):
    bit = torch.arange(32, device=mask.device)
    return (((mask.long()[:, :, None] >> bit) & 1) != 0).reshape(mask.shape[0], -1)


def _plain_mask(s):
    c, dev, t = s["case"], s["cu_q"].device, s["tokens_total"]
    seen = _dense_mask(s)
    count = s["cu_q"][1:] - s["cu_q"][:-1]
    req = torch.repeat_interleave(torch.arange(c["n"], device=dev), count.long(), output_size=t)
    depth = torch.where(count[req] <= 32 * _words(c), seen.sum(1) - 1, torch.arange(t, device=dev) - s["cu_q"][req])
    return _pack(seen, _words(c)), ((s["kv_len"] - count)[req] + depth).to(torch.int32)


def _plain_tree(s, mask):
    """One request after another, a block of its queries at a time (so that the scores fit)."""
    c, ps = s["case"], s["case"]["page"]
    hk, g, d = c["kv_heads"], c["heads"] // c["kv_heads"], c["head_dim"]
    o, lse = torch.empty_like(s["o"]), torch.empty_like(s["lse"])
    bits = _unpack(mask)
    for b, (q_len, kv) in enumerate(zip(s["new"], s["total"])):
        t0 = s["cu"][b]
        at = s["table"][b, : -(-kv // ps)].long()
        k, v = (x[at].transpose(0, 1).reshape(hk, -1, d)[:, :kv].float() for x in (s["k_cache"], s["v_cache"]))
        keys = torch.arange(kv, device=k.device)
        step = max(1, (1 << 28) // (c["heads"] * kv))
        for r0 in range(0, q_len, step):
            r1 = min(q_len, r0 + step)
            rows = s["q"][t0 + r0 : t0 + r1].float().view(r1 - r0, hk, g, d).permute(1, 2, 0, 3)  # [kv heads, group, rows, d]
            seen = keys[None] <= torch.arange(kv - q_len + r0, kv - q_len + r1, device=k.device)[:, None]
            if q_len <= 32 * _words(c):
                seen[:, kv - q_len :] &= bits[t0 + r0 : t0 + r1, :q_len]
            x = torch.matmul(rows.reshape(hk, g * (r1 - r0), d), k.transpose(-1, -2)) * d ** -0.5
            x = torch.where(seen.repeat(g, 1), x, -math.inf)
            m = x.amax(-1, keepdim=True)
            m = torch.where(torch.isinf(m), 0.0, m)
            e = torch.exp(x - m)
            norm = e.sum(-1, keepdim=True)
            y = torch.matmul(e, v) / torch.where(norm == 0, 1.0, norm)
            o[t0 + r0 : t0 + r1] = y.view(hk, g, r1 - r0, d).permute(2, 0, 1, 3).reshape(r1 - r0, hk * g, d)
            lse[:, t0 + r0 : t0 + r1] = (m + torch.log(norm)).view(hk * g, r1 - r0)
    return o, lse


def _plain_verify(s):
    """Every request at once, node by node in order: a node whose parent is the last one kept is tried.  In 64 bits:
    sums over a vocabulary are compared with a random number."""
    c, dev = s["case"], s["cu_q"].device
    n, v = c["n"], c["vocab"]
    some = lambda x: torch.where((x > 0) & (x < math.inf), x, 0.0).double()  # noqa: E731
    first, nodes = s["cu_q"][:-1].long(), (s["cu_q"][1:] - s["cu_q"][:-1]).long()
    every = torch.arange(n, device=dev)
    cur, kept = torch.zeros(n, dtype=torch.long, device=dev), torch.ones(n, dtype=torch.long, device=dev)
    a, mass = torch.zeros(n, dtype=torch.float64, device=dev), torch.ones(n, dtype=torch.float64, device=dev)
    gone = None if c["drafted"] else torch.zeros((n, v), dtype=torch.bool, device=dev)
    path = torch.full((n, s["width"]), -1, dtype=torch.long, device=dev)
    path[:, 0] = 0
    for t in range(1, max(s["new"])):
        at = torch.clamp(first + t, max=s["tokens_total"] - 1)
        row, x = first + cur, s["node_tokens"][at].long()
        tried = (t < nodes) & (s["parent"][at] == cur) & (kept < s["width"])
        p, u = some(s["target"][row, x]), s["u"][at].double()
        if c["drafted"]:
            q = some(s["draft"][row, x])
            yes = tried & (u * q * mass < (p - a * q).clamp(min=0))
            no = tried & ~yes
            a2 = a + mass
            mass2 = (some(s["target"][row]) - a2[:, None] * some(s["draft"][row])).clamp(min=0).sum(1)
            a = torch.where(no, torch.where(mass2 > 0, a2, 0.0), torch.where(yes, 0.0, a))
            mass = torch.where(no & (mass2 > 0), mass2, torch.where(yes | no, 1.0, mass))
        else:
            p = torch.where(gone[every, x], 0.0, p)
            yes = tried & (u * mass < p)
            no = tried & ~yes
            gone[every, x] |= no
            gone &= ~yes[:, None]
            mass = torch.where(no, (mass - p).clamp(min=0), torch.where(yes, 1.0, mass))
        path[every, torch.where(yes, kept, 0)] = torch.where(yes, t, path[:, 0])
        cur, kept = torch.where(yes, t, cur), kept + yes
    rows = some(s["target"][first + cur])
    if c["drafted"]:
        left = (rows - a[:, None] * some(s["draft"][first + cur])).clamp(min=0)
    else:
        left = torch.where(gone, 0.0, rows)
        left = torch.where(left.sum(1, keepdim=True) > 0, left, rows)
    upto = left.cumsum(1)
    nxt = (upto <= s["u_last"].double()[:, None] * upto[:, -1:]).sum(1)
    last = v - 1 - (left.flip(1) > 0).int().argmax(1)  # the last token with any mass
    nxt = torch.where(upto[:, -1] > 0, torch.minimum(nxt, last), -1)
    return path.to(torch.int32), kept.to(torch.int32), nxt.to(torch.int32)


def _plain_write(s):
    ps = s["case"]["page"]
    s["k_cache"][s["slots"] // ps, :, s["slots"] % ps] = s["k"]
    s["v_cache"][s["slots"] // ps, :, s["slots"] % ps] = s["v"]


def _plain_keep(s, path, kept):
    """Lengths, the list of free pages, and the rows of the kept nodes moved behind the keys that were there."""
    c, ps, dev = s["case"], s["case"]["page"], s["cu_q"].device
    n, new, kv = c["n"], (s["cu_q"][1:] - s["cu_q"][:-1]).long(), s["kv_len"].long()
    stay = torch.where(kept < 0, new, kept.long())
    out = kv - new + stay
    have, want = (kv + ps - 1) // ps, (out + ps - 1) // ps
    j = torch.arange(s["table"].shape[1], device=dev)
    give = (j >= want[:, None]) & (j < have[:, None])
    free, count = torch.cat([s["free"], s["free"][:1]]), s["count"].long()  # (its last entry takes what is not given back)
    rank = torch.where(give.reshape(-1), give.reshape(-1).cumsum(0) - 1 + count, free.numel() - 1)
    free = free.scatter(0, rank, s["table"].reshape(-1))[:-1]
    j = torch.arange(s["width"], device=dev)
    move = (j < kept[:, None]) & (path != j)
    slot = lambda pos: s["table"].gather(1, (pos // ps).clamp(0, s["table"].shape[1] - 1)).long() * ps + pos % ps  # noqa: E731
    base = (kv - new)[:, None]
    src, dst = slot(base + path.long().clamp(min=0)), slot(base + j)
    for cache in (s["k_cache"], s["v_cache"]):  # (a row that stays: the root's is put where it is)
        a, b = (torch.where(move, x, slot(base)).reshape(-1) for x in (src, dst))
        cache[b // ps, :, b % ps] = cache[a // ps, :, a % ps]
    return {"kv_len": out.to(torch.int32), "free": free, "count": (count + give.sum()).to(torch.int32),
            "src": torch.where(move, src, -1), "dst": torch.where(move, dst, -1)}


def _plain(s):
    kind, out = s["case"]["kind"], {}
    if kind in ("mask", "step"):
        out["mask"], out["positions"] = _plain_mask(s)
    if kind in ("keep", "step"):
        _plain_write(s)
    if kind in ("tree", "step"):
        out["o"], out["lse"] = _plain_tree(s, s["mask"] if kind == "tree" else out["mask"])
    if kind in ("verify", "step"):
        out["path"], out["kept"], out["next"] = _plain_verify(s)
    if kind in ("keep", "step"):
        src = out if kind == "step" else s
        out.update(_plain_keep(s, src["path"], src["kept"]), k_cache=s["k_cache"], v_cache=s["v_cache"])
    return out


# ---------------------------------------------------------------- the package's entry points
def _own(s):
    import fixed_max_softmax_gb300 as fm

    c, kind, out = s["case"], s["case"]["kind"], {}
    if kind in ("tree", "step") and "workspace" not in s:  # what a program keeps beside its buffers
        nbytes = fm.fm_attn_seqs_workspace_size(c["n"], s["tokens_total"], c["heads"], c["kv_heads"], c["head_dim"])
        s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        s["opts"] = fm.seqs_opts()
    if kind in ("mask", "step"):
        fm.fm_tree_mask(s["parent"], s["cu_q"], s["kv_len"], s["mask_out"], s["positions"])
        out.update(mask=s["mask_out"], positions=s["positions"])
    if kind in ("keep", "step"):
        fm.fm_paged_write(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"])
    if kind in ("tree", "step"):
        fm.fm_attn_tree(s["q"], s["k_cache"], s["v_cache"], s["cu_q"], s["kv_len"], s["table"],
                        s["mask"] if kind == "tree" else s["mask_out"], s["opts"], s["o"], s["lse"], s["workspace"])
        out.update(o=s["o"], lse=s["lse"])
    if kind in ("verify", "step"):
        fm.fm_tree_verify(s["target"], s["draft"], s["cu_q"], s["node_tokens"], s["parent"], s["u"], s["u_last"], s["path"],
                          s["kept"], s["next"])
        out.update(path=s["path"], kept=s["kept"], next=s["next"])
    if kind in ("keep", "step"):
        fm.fm_paged_keep(s["cu_q"], s["path"], s["kept"], s["kv_len"], s["kv_out"], s["table"], s["free"], s["count"],
                         s["count_out"], c["page"], s["src"], s["dst"], s["status"])
        fm.fm_paged_move(s["src"], s["dst"], s["k_cache"], s["v_cache"])
        out.update(kv_len=s["kv_out"], free=s["free"], count=s["count_out"], src=s["src"], dst=s["dst"], k_cache=s["k_cache"],
                   v_cache=s["v_cache"])
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64 bits, from the definition
def _exact_attention(c, s, kc, vc, out):
    ps, hk, d = c["page"], c["kv_heads"], c["head_dim"]
    group = c["heads"] // hk
    out["o"] = torch.zeros((s["tokens_total"], c["heads"], d), dtype=torch.float64, device="cuda")
    out["lse"] = torch.full((c["heads"], s["tokens_total"]), -math.inf, dtype=torch.float64, device="cuda")
    for i, (q, kv, parent, _) in enumerate(s["reqs"]):
        t, pages = s["cu"][i], s["table"][i, : -(-kv // ps)].long()
        k = kc[pages].transpose(1, 2).reshape(-1, hk, d)[:kv]
        v = vc[pages].transpose(1, 2).reshape(-1, hk, d)[:kv]
        hidden = torch.ones((q, q), dtype=torch.bool)  # among the new tokens
        for x, way in enumerate(_ancestors(parent) if parent else [list(range(x + 1)) for x in range(q)]):
            hidden[x, way] = False
        hidden = hidden.cuda()
        for h in range(c["heads"]):
            x = s["q"][t : t + q, h].double() @ k[:, h // group].T / math.sqrt(d)
            x[:, kv - q :][hidden] = -math.inf
            out["lse"][h, t : t + q] = torch.logsumexp(x, 1)
            out["o"][t : t + q, h] = torch.softmax(x, 1) @ v[:, h // group]


def _exact_walk(c, s, i):
    """One request's walk: (path, next token)."""
    first, (q, _, parent, _) = s["cu"][i], s["reqs"][i]
    tokens = s["node_tokens"][first : first + q].tolist()
    u, u_last = s["u"][first : first + q].tolist(), float(s["u_last"][i])
    path = [0]
    while True:
        at = path[-1]
        left, mass = s["target"][first + at].double().clone(), 1.0  # what is left of the target's row, and its mass
        draft = s["draft"][first + at].double() if c["drafted"] else None
        for t in [t for t in range(at + 1, q) if parent[t] == at]:
            x = tokens[t]
            if u[t] * mass * (1.0 if draft is None else float(draft[x])) < float(left[x]):
                path.append(t)
                break
            if draft is None:
                mass = max(mass - float(left[x]), 0.0)
                left[x] = 0.0
            else:
                left = (left - mass * draft).clamp(min=0)
                mass = float(left.sum())
                if mass == 0.0:
                    left, mass = s["target"][first + at].double().clone(), 1.0
        if path[-1] == at:
            break
    if float(left.sum()) == 0.0:
        left = s["target"][first + at].double()
    upto = left.cumsum(0)
    have = torch.nonzero(left).flatten()
    if not len(have):
        return path, -1
    return path, min(int((upto <= u_last * float(upto[-1])).sum()), int(have[-1]))


def exact(case, seed):
    c = case
    w = work(c)
    if c["kind"] == "mask" or (c["kind"] in ("tree", "step") and w["flops"] > 1e12):
        return None
    if c["kind"] == "verify" and c["n"] * c["nodes"] > 3000:
        return None
    s = prepare(case, seed)
    ps, out = c["page"], {}
    kc, vc = (s["k_cache"].double(), s["v_cache"].double()) if "table" in s else (None, None)
    if c["kind"] == "step":
        out.update(mask=None, positions=None)
    if c["kind"] in ("keep", "step"):
        for i, (q, kv, _, _) in enumerate(s["reqs"]):
            p = torch.arange(kv - q, kv, device="cuda")
            page, t = s["table"][i].long()[p // ps], s["cu"][i]
            kc[page, :, p % ps], vc[page, :, p % ps] = s["k"][t : t + q].double(), s["v"][t : t + q].double()
    if c["kind"] in ("tree", "step"):
        _exact_attention(c, s, kc, vc, out)
    paths = [r[3] for r in s["reqs"]]
    if c["kind"] in ("verify", "step"):
        walks = [_exact_walk(c, s, i) for i in range(c["n"])]
        paths = [p for p, _ in walks]
        whole = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        out.update(path=whole([p + [-1] * (s["width"] - len(p)) for p in paths]), kept=whole([len(p) for p in paths]),
                   next=whole([x for _, x in walks]))
    if c["kind"] in ("keep", "step"):
        out.update(kv_len=None, free=None, count=None, src=None, dst=None)
        for i, (q, kv, _, _) in enumerate(s["reqs"]):
            for j, x in enumerate(paths[i] or []):
                to, at = kv - q + j, kv - q + x
                for cache in (kc, vc):
                    cache[s["table"][i, to // ps], :, to % ps] = cache[s["table"][i, at // ps], :, at % ps]
        out.update(k_cache=kc, v_cache=vc)
    return out
