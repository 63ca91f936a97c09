"""The serving operators of this package as measured workloads.

    extend   fm_paged_extend: page tables, slot maps and positions of the next tokens of a batch of
             requests, built on the GPU from their lengths
    write    fm_paged_write: new key and value rows put into a paged cache at their slots
    paged    fm_attn_paged: attention of each request's new tokens (one, or a chunk) over its pages
    varlen   fm_attn_varlen: attention of whole prompts of different lengths, packed
    step     the three paged operators in a row, as one layer of a serving step runs them

`run` computes them in plain torch operations, or with `own` true through the package's entry
points.  Lengths are a function of the case alone (its `mix` seeds them), values of the seed.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


def _case(name, kind, **kw):
    c = {"kind": kind, "dtype": "bf16", "n": 1, "chunks": 0, "q_max": 1, "kv_max": 1024, "heads": 32, "kv_heads": 8,
         "head_dim": 128, "page": 16, "causal": True, "window": 0, "release": 0, "mix": 1, "token_major": True}
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the bookkeeping before each decode step of a small server: one new token per request
        _case("extend decode 48", "extend", n=48, kv_max=2000, mix=3),
        # a burst of long prompts admitted at once, while 9 finished requests give back their pages
        _case("extend prompts 96", "extend", n=96, chunks=90, q_max=8192, kv_max=9000, release=9, mix=4),
        # one layer's new keys and values of a decode batch
        _case("write decode 64", "write", n=64, kv_max=512, mix=5),
        # one layer's keys and values of a batch of prompts, 64-token pages, one page's head rows together
        _case("write prompts 65k", "write", n=24, chunks=24, q_max=4803, kv_max=4803, page=64, token_major=False, mix=6),
        # one user, one token, a short context: latency alone
        _case("decode one 777", "paged", n=1, kv_max=777, mix=7),
        # a full decode batch, contexts of all lengths, 5 query heads to a key head
        _case("decode batch 64", "paged", n=64, kv_max=8192, heads=40, mix=8),
        # few users with very long contexts: every key has to be streamed
        _case("decode long 131k", "paged", n=4, kv_max=131072, heads=64, page=64, dtype="fp16", token_major=False, mix=9),
        # chunked prefill beside decoding requests: chunks of up to 512 new tokens over contexts of up to 32k
        _case("chunks 512 over 32k", "paged", n=12, chunks=5, q_max=512, kv_max=32768, page=32, mix=10),
        # a handful of short prompts in full precision, as many key heads as query heads
        _case("prompts short fp32", "varlen", n=5, chunks=5, kv_max=201, heads=12, kv_heads=12, head_dim=64, dtype="fp32",
              mix=11),
        # a prefill batch of prompts of all lengths
        _case("prompts packed 4k", "varlen", n=24, chunks=24, kv_max=4096, heads=40, mix=12),
        # one very long prompt
        _case("prompt long 33k", "varlen", n=1, chunks=1, kv_max=33001, heads=40, mix=13),
        # a whole serving step of one layer: 120 decoding requests and 3 prompt chunks
        _case("step 123", "step", n=123, chunks=3, q_max=384, kv_max=4096, heads=40, mix=14),
    ]


def _between(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["extend", "write", "paged", "paged", "paged", "varlen", "varlen", "step"])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 10])
    group = rng.choice([1, 2, 4, 4, 5, 7, 8])
    c = _case(None, kind, mix=rng.randrange(1 << 20), kv_heads=kv_heads, heads=kv_heads * group,
              head_dim=rng.choice([64, 128, 128]), dtype=rng.choice(["bf16", "bf16", "bf16", "fp16", "fp16", "fp32"]),
              page=rng.choice([8, 16, 16, 32, 64, 128]), token_major=rng.random() < 0.5)
    if kind == "varlen":
        if c["dtype"] == "fp32":
            c.update(n=_between(rng, 1, 6), kv_max=_between(rng, 16, 400))
        else:
            c.update(n=_between(rng, 1, 32), kv_max=_between(rng, 16, 8000))
        c.update(chunks=c["n"], causal=rng.random() < 0.85, page=16)
    elif kind == "extend":
        c.update(n=_between(rng, 1, 256), kv_max=_between(rng, 64, 9000))
        c.update(chunks=rng.randint(0, c["n"]), q_max=_between(rng, 1, c["kv_max"]), release=rng.randint(0, c["n"] // 4))
    elif kind == "write":
        c.update(n=_between(rng, 1, 64), kv_max=_between(rng, 16, 4000))
        c.update(chunks=rng.randint(0, c["n"]), q_max=_between(rng, 1, c["kv_max"]))
    else:
        c.update(n=_between(rng, 1, 128), kv_max=_between(rng, 100, 32000 if kind == "paged" else 6000))
        while c["n"] * c["kv_max"] > 600000:
            c["n"] = (c["n"] + 1) // 2
        if rng.random() < 0.5 and c["dtype"] != "fp32":
            c.update(chunks=rng.randint(1, min(4, c["n"])), q_max=_between(rng, 2, min(700, c["kv_max"])))
    if c["causal"] and kind in ("paged", "varlen") and rng.random() < 0.25:
        c["window"] = _between(rng, 16, 4096)
    return c


def _lengths(c):
    """(new tokens, keys with the new ones) of each request; the first has the case's largest."""
    rng = random.Random(c["mix"])
    new, total = [], []
    for i in range(c["n"]):
        many = i < c["chunks"]
        if c["kind"] == "varlen":
            s = c["kv_max"] if i == 0 else _between(rng, max(1, c["kv_max"] // 16), c["kv_max"])
            new.append(s)
            total.append(s)
            continue
        q = 1 if not many else c["q_max"] if i == 0 else _between(rng, max(1, c["q_max"] // 8), c["q_max"])
        s = c["kv_max"] if i == 0 else _between(rng, max(1, c["kv_max"] // 16), c["kv_max"])
        new.append(q)
        total.append(max(q, s))
    return new, total


def _pairs(c):
    """(query, key) pairs that are seen, and the keys that any query of their request sees."""
    pairs = keys = 0
    for q, s in zip(*_lengths(c)):
        if not c["causal"]:
            pairs += q * s
            keys += s
            continue
        w = c["window"] or s
        first = s - q  # position of the first query; it sees min(first + 1, w) keys
        ramp = max(0, min(q, w - first - 1))  # queries that see fewer than w keys
        pairs += ramp * (first + 1) + ramp * (ramp - 1) // 2 + (q - ramp) * w
        keys += s - max(0, first + 1 - w)
    return pairs, keys


def work(case):
    c, es = case, BYTES[case["dtype"]]
    new, total = _lengths(c)
    t, n = sum(new), c["n"]
    row = c["kv_heads"] * c["head_dim"] * es
    pages = sum(-(-s // c["page"]) for s in total)
    old_pages = sum(-(-(s - q) // c["page"]) for q, s in zip(new, total))
    back = sum(-(-total[n - 1 - i] // c["page"]) for i in range(c["release"]))
    # lengths, new pages from the list into the table, pages given back, a slot and a position per token, the page
    # that each request's first new token may share with its old ones
    extend = 4 * (4 * n + 1) + n + 8 * (pages - old_pages + back) + 12 * t + 4 * n
    write = 4 * t * row + 8 * t
    if c["kind"] == "extend":
        return {"bytes": extend, "flops": 0}
    if c["kind"] == "write":
        return {"bytes": write, "flops": 0}
    pairs, keys = _pairs(c)
    attn = 2 * t * c["heads"] * c["head_dim"] * es + 4 * t * c["heads"] + 2 * keys * row + 8 * n
    if c["kind"] != "varlen":
        attn += 4 * -(-keys // c["page"])
    flops = 4.0 * pairs * c["heads"] * c["head_dim"]
    return {"bytes": attn + (extend + write if c["kind"] == "step" else 0), "flops": flops}


def _cache_of(c, pages, make):
    shape = (pages, c["page"], c["kv_heads"], c["head_dim"]) if c["token_major"] else (
        pages, c["kv_heads"], c["page"], c["head_dim"])
    t = make(shape)
    return t.transpose(1, 2) if c["token_major"] else t  # [pages, kv heads, page, head dim] either way


def prepare(case, seed):
    c, dt, dev = case, DTYPES[case["dtype"]], "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    rand = lambda *shape: torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dt)  # noqa: E731
    new, total = _lengths(c)
    n, t = c["n"], sum(new)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    cu = [0]
    for q in new:
        cu.append(cu[-1] + q)
    s = {"case": c, "new": new, "total": total, "tokens": t, "cu_q": ints(cu)}
    if c["kind"] in ("paged", "varlen", "step"):
        # heads look with different sharpness
        sharp = torch.rand((c["heads"], 1), generator=g, device=dev) * 1.5 + 0.5
        s["q"] = (torch.randn((t, c["heads"], c["head_dim"]), generator=g, device=dev) * sharp).to(dt)
        s["o"] = torch.empty((t, c["heads"], c["head_dim"]), dtype=dt, device=dev)
        s["lse"] = torch.empty((c["heads"], t), dtype=torch.float32, device=dev)
    if c["kind"] in ("write", "step", "varlen"):
        s["k"], s["v"] = rand(t, c["kv_heads"], c["head_dim"]), rand(t, c["kv_heads"], c["head_dim"])
    if c["kind"] == "varlen":
        s["cu_k"] = s["cu_q"].clone()
        return s
    # a cache with every page that the requests need and some more, its pages dealt out in random order
    ps = c["page"]
    need = [-(-x // ps) for x in total]
    held = need if c["kind"] in ("paged", "write") else [-(-(x - q) // ps) for q, x in zip(new, total)]
    if c["kind"] == "extend":  # the requests that end: they hold all their pages and get no new tokens
        new, held = list(new), list(held)
        for i in range(c["release"]):
            new[n - 1 - i], held[n - 1 - i] = 0, need[n - 1 - i]
        s["tokens"] = t = sum(new)
    pages = sum(need) + sum(need) // 8 + 16
    order = torch.randperm(pages, generator=g, device=dev, dtype=torch.int64).to(torch.int32)
    width = max(need) + 1
    table = torch.full((n, width), -1, dtype=torch.int32, device=dev)
    req = torch.repeat_interleave(torch.arange(n, device=dev), torch.tensor(held, device=dev))
    start = torch.tensor([sum(held[:i]) for i in range(n)], device=dev)
    table[req, torch.arange(sum(held), device=dev) - start[req]] = order[: sum(held)]
    s.update(table=table, pages=pages)
    if c["kind"] in ("extend", "step"):
        released = [i >= n - c["release"] for i in range(n)] if c["kind"] == "extend" else [False] * n
        s["new_len"] = ints(new)
        s["release"] = torch.tensor(released, dtype=torch.uint8, device=dev)
        s["kv_len"] = ints([x if r else x - q for x, q, r in zip(total, new, released)])
        s["kv_out"] = torch.empty(n, dtype=torch.int32, device=dev)
        free = pages - sum(held)
        s["free"] = torch.full((pages,), -1, dtype=torch.int32, device=dev)
        s["free"][:free] = order[sum(held):]
        s["count"], s["count_out"] = ints([free]), ints([0])
        s["slots"] = torch.empty(t, dtype=torch.int64, device=dev)
        s["positions"] = torch.empty(t, dtype=torch.int32, device=dev)
        s["status"] = ints([0])
        # what the program that admits requests knows of them: pages given back and new pages
        s["back"] = sum(h for h, r in zip(held, released) if r)
        s["fresh"] = sum(0 if r else a - h for a, h, r in zip(need, held, released))
    if c["kind"] == "paged":
        s["kv_len"] = ints(total)
    if c["kind"] == "write":  # slots of the last `new` positions of each request
        req = torch.repeat_interleave(torch.arange(n, device=dev), torch.tensor(new, device=dev))
        pos = torch.arange(t, device=dev) - s["cu_q"][req] + (torch.tensor(total, device=dev) - torch.tensor(new, device=dev))[req]
        s["slots"] = table[req, pos // ps].long() * ps + pos % ps
    if c["kind"] != "extend":
        s["k_cache"] = _cache_of(c, pages, lambda shape: rand(*shape))
        s["v_cache"] = _cache_of(c, pages, lambda shape: rand(*shape))
    return s


# ---------------------------------------------------------------- plain forms
def _plain_extend(s):
    """Pages given back go on top of the list in request order, new pages come off its top."""
    c, ps, dev = s["case"], s["case"]["page"], s["table"].device
    n, t, back, fresh = c["n"], s["tokens"], s["back"], s["fresh"]
    at = torch.arange(n, device=dev)
    new, out = s["new_len"].long(), s["release"].bool()
    old_pages = (s["kv_len"].long() + ps - 1) // ps
    base = torch.where(out, 0, s["kv_len"].long())
    base_pages = (base + ps - 1) // ps
    count = s["count"].long()
    free, table = s["free"].clone(), s["table"].clone()
    given = torch.where(out, old_pages, 0)
    req = torch.repeat_interleave(at, given, output_size=back)
    run_ = torch.arange(back, device=dev)
    free[count + run_] = table[req, run_ - (given.cumsum(0) - given)[req]]
    want = (base + new + ps - 1) // ps - base_pages
    req = torch.repeat_interleave(at, want, output_size=fresh)
    run_ = torch.arange(fresh, device=dev)
    table[req, base_pages[req] + run_ - (want.cumsum(0) - want)[req]] = free[count + back - 1 - run_]
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), new.cumsum(0)])
    req = torch.repeat_interleave(at, new, output_size=t)
    pos = base[req] + torch.arange(t, device=dev) - cu[req]
    slots = table[req, pos // ps].long() * ps + pos % ps
    return {"cu_q": cu.int(), "slots": slots, "positions": pos.int(), "kv_len": (base + new).int(), "table": table,
            "free": free, "count": (count + back - fresh).int()}


def _plain_write(s, slots):
    ps = s["case"]["page"]
    s["k_cache"][slots // ps, :, slots % ps] = s["k"]
    s["v_cache"][slots // ps, :, slots % ps] = s["v"]


def _plain_softmax(q, k, v, seen, scale):
    """softmax(scale q k^T) v over the seen keys, and its log-sum-exp; a row that sees none gives zeros."""
    x = torch.where(seen, torch.matmul(q, k.transpose(-1, -2)) * scale, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(m), 0.0, m))
    total = e.sum(-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(total == 0, 1.0, total)
    return o, (m + torch.log(total)).squeeze(-1)


def _plain_seen(c, pos, keys):
    if not c["causal"]:
        return torch.ones((pos.numel(), keys.numel()), dtype=torch.bool, device=pos.device)
    seen = keys[None] <= pos[:, None]
    return seen & (keys[None] > pos[:, None] - c["window"]) if c["window"] else seen


def _plain_attention(s, keys_of, total):
    """One request after another, a block of its queries at a time (so that the scores fit)."""
    c = s["case"]
    hk, g, d = c["kv_heads"], c["heads"] // c["kv_heads"], c["head_dim"]
    o, lse = torch.empty_like(s["o"]), torch.empty_like(s["lse"])
    t0 = 0
    for b, (q_len, kv) in enumerate(zip(s["new"], total)):
        k, v = keys_of(b, kv)  # [kv heads, keys, head dim] in 32 bits
        at = torch.arange(kv, device=k.device)
        step = max(1, (1 << 29) // (c["heads"] * kv))
        for r0 in range(0, q_len, step):
            r1 = min(q_len, r0 + step)
            rows = s["q"][t0 + r0 : t0 + r1].float().view(r1 - r0, hk, g, d).permute(1, 2, 0, 3)  # [kv heads, group, rows, d]
            seen = _plain_seen(c, torch.arange(kv - q_len + r0, kv - q_len + r1, device=k.device), at)
            y, z = _plain_softmax(rows.reshape(hk, g * (r1 - r0), d), k, v, seen.repeat(g, 1), d ** -0.5)
            o[t0 + r0 : t0 + r1] = y.view(hk, g, r1 - r0, d).permute(2, 0, 1, 3).reshape(r1 - r0, hk * g, d)
            lse[:, t0 + r0 : t0 + r1] = z.view(hk * g, r1 - r0)
        t0 += q_len
    return o, lse


def _plain_decode(s, table, kv_len):
    """One token per request: every request at once, padded to the longest."""
    c, ps = s["case"], s["case"]["page"]
    n, hk, g, d = c["n"], c["kv_heads"], c["heads"] // c["kv_heads"], c["head_dim"]
    width = -(-max(s["total"]) // ps)
    at = table[:, :width].clamp(min=0).long()
    gather = lambda x: x[at].permute(0, 2, 1, 3, 4).reshape(n, hk, width * ps, d).float()  # noqa: E731
    keys = torch.arange(width * ps, device=table.device)
    seen = keys[None] < kv_len[:, None]
    if c["window"]:
        seen = seen & (keys[None] >= kv_len[:, None] - c["window"])
    o, lse = _plain_softmax(s["q"].float().view(n, hk, g, d), gather(s["k_cache"]), gather(s["v_cache"]), seen[:, None, None],
                            d ** -0.5)
    return o.reshape(n, hk * g, d).to(s["q"].dtype), lse.reshape(n, hk * g).t().contiguous()


def _plain_paged(s, table, kv_len):
    c, ps = s["case"], s["case"]["page"]
    if s["tokens"] == c["n"]:
        return _plain_decode(s, table, kv_len)

    def keys_of(b, kv):
        at = table[b, : -(-kv // ps)].long()
        flat = lambda x: x[at].transpose(0, 1).reshape(c["kv_heads"], -1, c["head_dim"])[:, :kv].float()  # noqa: E731
        return flat(s["k_cache"]), flat(s["v_cache"])

    return _plain_attention(s, keys_of, s["total"])


def _plain(s):
    c = s["case"]
    if c["kind"] == "extend":
        return _plain_extend(s)
    if c["kind"] == "write":
        _plain_write(s, s["slots"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if c["kind"] == "paged":
        o, lse = _plain_paged(s, s["table"], s["kv_len"])
        return {"o": o, "lse": lse}
    if c["kind"] == "varlen":
        at = [0]
        for x in s["total"]:
            at.append(at[-1] + x)
        keys_of = lambda b, kv: (s["k"][at[b] : at[b] + kv].transpose(0, 1).float(), s["v"][at[b] : at[b] + kv].transpose(0, 1).float())  # noqa: E731
        o, lse = _plain_attention(s, keys_of, s["total"])
        return {"o": o, "lse": lse}
    r = _plain_extend(s)
    _plain_write(s, r["slots"])
    o, lse = _plain_paged(s, r["table"], r["kv_len"])
    return {"slots": r["slots"], "kv_len": r["kv_len"], "table": r["table"], "o": o, "lse": lse, "k_cache": s["k_cache"],
            "v_cache": s["v_cache"]}


# ---------------------------------------------------------------- the package's entry points
def _own(s):
    import fixed_max_softmax_gb300 as fm

    c = s["case"]
    if c["kind"] in ("paged", "varlen", "step") and "workspace" not in s:  # what a program keeps beside its buffers
        nbytes = fm.fm_attn_seqs_workspace_size(c["n"], s["tokens"], c["heads"], c["kv_heads"], c["head_dim"])
        s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        s["opts"] = fm.seqs_opts(causal=c["causal"], window=c["window"])
    if c["kind"] in ("extend", "step"):
        fm.fm_paged_extend(s["new_len"], s["release"], s["kv_len"], s["kv_out"], s["table"], s["free"], s["count"],
                           s["count_out"], c["page"], s["cu_q"], s["slots"], s["positions"], s["status"])
    if c["kind"] == "extend":
        return {"cu_q": s["cu_q"], "slots": s["slots"], "positions": s["positions"], "kv_len": s["kv_out"],
                "table": s["table"], "free": s["free"], "count": s["count_out"]}
    if c["kind"] in ("write", "step"):
        fm.fm_paged_write(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"])
    if c["kind"] == "write":
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if c["kind"] == "varlen":
        fm.fm_attn_varlen(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["opts"], s["o"], s["lse"], s["workspace"])
        return {"o": s["o"], "lse": s["lse"]}
    kv_len = s["kv_out"] if c["kind"] == "step" else s["kv_len"]
    fm.fm_attn_paged(s["q"], s["k_cache"], s["v_cache"], s["cu_q"], kv_len, s["table"], s["opts"], s["o"], s["lse"],
                     s["workspace"])
    if c["kind"] == "paged":
        return {"o": s["o"], "lse": s["lse"]}
    return {"slots": s["slots"], "kv_len": s["kv_out"], "table": s["table"], "o": s["o"], "lse": s["lse"],
            "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- 64 bits, from the definition
def exact(case, seed):
    c = case
    if c["kind"] == "extend" or work(c)["flops"] > 1.2e12:
        return None
    s = prepare(c, seed)
    ps, hk, d = c["page"], c["kv_heads"], c["head_dim"]
    group = c["heads"] // hk
    out = {}
    table = s["table"].tolist() if "table" in s else None
    if c["kind"] == "step":  # the new pages come off the end of the list, one request after another
        free = s["free"][: int(s["count"])].tolist()
        for i, (q, kv) in enumerate(zip(s["new"], s["total"])):
            for j in range(-(-(kv - q) // ps), -(-kv // ps)):
                table[i][j] = free.pop()
        out.update(slots=None, kv_len=None, table=None)
    kc, vc = (s["k_cache"].double(), s["v_cache"].double()) if table is not None else (None, None)
    if c["kind"] in ("write", "step"):
        t = 0
        for i, (q, kv) in enumerate(zip(s["new"], s["total"])):
            p = torch.arange(kv - q, kv, device="cuda")
            page = torch.tensor(table[i], device="cuda")[p // ps]
            kc[page, :, p % ps] = s["k"][t : t + q].double()
            vc[page, :, p % ps] = s["v"][t : t + q].double()
            t += q
        out.update(k_cache=kc, v_cache=vc)
        if c["kind"] == "write":
            return out
    o = torch.zeros((s["tokens"], c["heads"], d), dtype=torch.float64, device="cuda")
    lse = torch.full((c["heads"], s["tokens"]), -math.inf, dtype=torch.float64, device="cuda")
    t = 0
    for i, (q, kv) in enumerate(zip(s["new"], s["total"])):
        if table is None:
            k, v = s["k"][t : t + kv].double(), s["v"][t : t + kv].double()
        else:
            pages = torch.tensor(table[i][: -(-kv // ps)], device="cuda")
            k = kc[pages].transpose(1, 2).reshape(-1, hk, d)[:kv]
            v = vc[pages].transpose(1, 2).reshape(-1, hk, d)[:kv]
        j = torch.arange(kv, device="cuda")
        step = max(1, (1 << 27) // kv)
        for h in range(c["heads"]):
            for r in range(0, q, step):
                e = min(q, r + step)
                x = s["q"][t + r : t + e, h].double() @ k[:, h // group].T / math.sqrt(d)
                if c["causal"]:
                    back = torch.arange(kv - q + r, kv - q + e, device="cuda")[:, None] - j  # how far back a key lies
                    x[(back < 0) | (back >= (c["window"] or kv + 1))] = -math.inf
                lse[h, t + r : t + e] = torch.logsumexp(x, 1)
                o[t + r : t + e, h] = torch.softmax(x, 1) @ v[:, h // group]
        t += q
    out.update(o=o, lse=lse)
    return out
