"""The attention block's operators between two fused all-reduce calls, as a user's program calls them.

Three operators of one serving step: the paged plan (block tables and slot maps from request lengths), the per-head norm with
rotation and cache write, and the attention of the new tokens over the paged cache.  `run` computes them in plain torch
operations, or through the framework where `own` is true; `exact` is the definition in 64 bits."""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # decode step of eight chat requests: one new token each, the smallest plan
        {"name": "plan decode 8", "kind": "plan", "requests": 8, "new": 1, "ctx": 4000, "mode": "ragged", "page": 16, "spare": 0, "lengths": 1},
        # a scheduler's step with chunks of 64 requests and 192 single tokens, padded for a captured graph
        {"name": "plan mixed 256", "kind": "plan", "requests": 256, "new": 512, "ctx": 9000, "mode": "mixed", "page": 16, "spare": 777, "lengths": 2},
        # an offline batch that is filled at once: 1024 prompts
        {"name": "plan prompts 1024", "kind": "plan", "requests": 1024, "new": 250, "ctx": 0, "mode": "ragged", "page": 64, "spare": 0, "lengths": 3},
        # decode of 16 requests (the benchmark's decode rows), 12 + 2 + 2 heads of 128 (6144 split over four ranks)
        {"name": "rope decode 16", "kind": "rope", "dtype": "bf16", "tokens": 16, "q_heads": 12, "kv_heads": 2, "head_dim": 128, "rot": 128,
         "pairs": False, "axes": 1, "dealt": False, "norm": True, "gemma": False, "far": 40000, "page": 16, "skip": 0},
        # the benchmark's 2800 rows of 6144 with all 48 + 8 + 8 heads, gemma weights, half of each head rotated
        {"name": "rope 2800 half", "kind": "rope", "dtype": "bf16", "tokens": 2800, "q_heads": 48, "kv_heads": 8, "head_dim": 128, "rot": 64,
         "pairs": False, "axes": 1, "dealt": False, "norm": True, "gemma": True, "far": 130000, "page": 16, "skip": 5},
        # image and video tokens with three position axes, frequencies dealt to the axes in turn, adjacent pairs, fp16, 80-wide heads
        {"name": "rope video 16384", "kind": "rope", "dtype": "fp16", "tokens": 16384, "q_heads": 16, "kv_heads": 16, "head_dim": 80, "rot": 80,
         "pairs": True, "axes": 3, "dealt": True, "norm": True, "gemma": False, "far": 2000, "page": 64, "skip": 0},
        # one request answers alone: latency
        {"name": "attend one token", "kind": "attend", "dtype": "bf16", "q_heads": 12, "kv_heads": 2, "head_dim": 128, "page": 16, "requests": 1,
         "new": 1, "ctx": 700, "mode": "each", "causal": True, "window": 0, "cap": 0.0, "slopes": False, "prefix": 0, "spare": 0, "lengths": 4},
        # decode of a full batch with ragged long contexts: bound by reading the cache
        {"name": "attend decode 64", "kind": "attend", "dtype": "bf16", "q_heads": 48, "kv_heads": 8, "head_dim": 128, "page": 16, "requests": 64,
         "new": 1, "ctx": 9000, "mode": "ragged", "causal": True, "window": 0, "cap": 0.0, "slopes": False, "prefix": 0, "spare": 3, "lengths": 5},
        # a chunk of a long prompt together with the others' single tokens, scores capped, sliding window, fp16, heads of 64
        {"name": "attend mixed window", "kind": "attend", "dtype": "fp16", "q_heads": 16, "kv_heads": 4, "head_dim": 64, "page": 32, "requests": 17,
         "new": 700, "ctx": 5000, "mode": "mixed", "causal": True, "window": 1024, "cap": 30.0, "slopes": False, "prefix": 0, "spare": 0, "lengths": 6},
        # prompts with a prefix that sees itself both ways and a bias by distance, 96-wide heads
        {"name": "attend prefix bias", "kind": "attend", "dtype": "bf16", "q_heads": 8, "kv_heads": 8, "head_dim": 96, "page": 64, "requests": 6,
         "new": 1500, "ctx": 0, "mode": "ragged", "causal": True, "window": 0, "cap": 0.0, "slopes": True, "prefix": 256, "spare": 0, "lengths": 7},
        # one key head of 256, a chunk over a middle context
        {"name": "attend wide heads", "kind": "attend", "dtype": "bf16", "q_heads": 8, "kv_heads": 1, "head_dim": 256, "page": 16, "requests": 2,
         "new": 1024, "ctx": 8000, "mode": "each", "causal": True, "window": 0, "cap": 0.0, "slopes": False, "prefix": 0, "spare": 0, "lengths": 8},
        # a 4096-row chunk (the benchmark's largest) of a long document: bound by the products
        {"name": "attend chunk 4096", "kind": "attend", "dtype": "bf16", "q_heads": 12, "kv_heads": 2, "head_dim": 128, "page": 64, "requests": 1,
         "new": 4096, "ctx": 28000, "mode": "each", "causal": True, "window": 0, "cap": 0.0, "slopes": False, "prefix": 0, "spare": 0, "lengths": 9},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["plan", "rope", "rope", "attend", "attend", "attend"])
    lengths = rng.randrange(1, 1 << 20)
    if kind == "plan":
        requests, mode = _log(rng, 1, 1024), rng.choice(["ragged", "mixed", "each"])
        new = max(1, min(_log(rng, 1, 2000), 250000 // requests))
        return {"kind": "plan", "requests": requests, "new": new, "ctx": rng.choice([0, _log(rng, 1, 9000)]), "mode": mode,
                "page": rng.choice([1, 8, 16, 24, 32, 64, 128]), "spare": rng.choice([0, _log(rng, 1, 1000)]), "lengths": lengths}
    dtype = rng.choice(["bf16", "fp16"])
    q_heads, kv_heads = rng.choice([(12, 2), (6, 1), (48, 8), (8, 8), (16, 4), (8, 1), (16, 16), (20, 4), (7, 1)])
    if kind == "rope":
        head_dim = rng.choice([64, 80, 96, 128, 256])
        most = 16384 * 48 * 80 // ((q_heads + 2 * kv_heads) * head_dim)
        rot = rng.choice([head_dim, head_dim, head_dim // 2, 2 * (head_dim // 8)])
        axes = rng.choice([1, 1, 2, 3, 4])
        return {"kind": "rope", "dtype": dtype, "tokens": _log(rng, 1, most), "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "rot": rot,
                "pairs": rng.random() < 0.4, "axes": axes, "dealt": axes > 1 and rng.random() < 0.5, "norm": rng.random() < 0.8, "gemma": rng.random() < 0.3,
                "far": _log(rng, 100, 1000000), "page": rng.choice([8, 16, 32, 64]), "skip": rng.choice([0, 0, 3])}
    head_dim = rng.choice([64, 80, 96, 128, 128, 128, 256])
    mode, requests = rng.choice(["ragged", "mixed", "each"]), _log(rng, 1, 64)
    ctx = rng.choice([0, _log(rng, 1, 24000), _log(rng, 1, 24000)])
    if rng.random() < 0.4:
        new, ctx = rng.choice([1, 1, 2, 5]), max(ctx, 40)
    else:  # the padded score matrix of the plain form stays below the largest listed case's
        new = _log(rng, 8, 3000)
        while requests * q_heads * new * (new + ctx) * head_dim > 1.5e11:
            requests, new, ctx = max(1, requests // 2), max(1, new * 3 // 4), ctx * 3 // 4
    while requests * (new + ctx) * kv_heads * head_dim > 5e8:
        requests, ctx = max(1, requests // 2), ctx * 3 // 4
    return {"kind": "attend", "dtype": dtype, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": rng.choice([8, 16, 32, 64, 128, 24]),
            "requests": requests, "new": new, "ctx": ctx, "mode": mode, "causal": rng.random() < 0.85, "window": rng.choice([0, 0, 0, _log(rng, 1, 4096)]),
            "cap": rng.choice([0.0, 0.0, 0.0, 20.0, 50.0]), "slopes": rng.random() < 0.2, "prefix": rng.choice([0, 0, 0, _log(rng, 1, 600)]),
            "spare": rng.choice([0, 0, 5]), "lengths": lengths}


def _lens(c):
    """(tokens in the cache, new tokens) of each request: fixed by the case."""
    rng, n, x = random.Random(c["lengths"]), c["new"], c["ctx"]
    if c["mode"] == "each":
        return [x] * c["requests"], [n] * c["requests"]
    if c["mode"] == "ragged":
        return [rng.randint(x // 4, x) for _ in range(c["requests"])], [rng.randint(-(-n // 4), n) for _ in range(c["requests"])]
    new = [n if i % 16 == 0 else 1 if i % 16 < 15 else 0 for i in range(c["requests"])]  # chunks, single tokens, some that wait
    return [rng.randint(x // 4, x) for _ in new], new


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _pages(c, cached, g):
    """A shuffled pool of blocks, each request's table row as far as its first `cached` tokens, and the free list."""
    p = c["page"]
    have, need = [-(-x // p) for x in cached], [-(-(x + n) // p) for x, n in zip(cached, _lens(c)[1])]
    total = sum(need) + 8 + sum(need) // 16
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    width = max(max(need), 1) + 3
    table = torch.full((c["requests"], width), -1, dtype=torch.int32, device="cuda")
    col = torch.arange(width, device="cuda")
    h = torch.tensor(have, device="cuda")
    first = torch.cumsum(h, 0) - h
    place = (first[:, None] + col).clamp(max=total - 1)
    table = torch.where(col < h[:, None], order[place], table)
    return table.contiguous(), order[sum(have):].contiguous(), total


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["kind"] == "plan":
        cached, new = _lens(c)
        table, free, total = _pages(c, cached, g)
        tokens = sum(new) + c["spare"]
        e = lambda n, t=torch.int32: torch.empty(n, dtype=t, device="cuda")  # noqa: E731
        # another seed shifts the lengths within their last page, as another step's requests would
        shift = torch.randint(0, 2, (c["requests"],), generator=g, device="cuda", dtype=torch.int32)
        length = _ints(cached)
        length = torch.where(length % c["page"] > 1, length - shift, length)
        return {"case": c, "cached": length, "new": _ints(new), "free": free, "count": _ints([free.numel()]), "table": table, "page": c["page"],
                "out": {"cu": e(c["requests"] + 1), "lens": e(c["requests"]), "slots": e(tokens, torch.int64), "positions": e(tokens), "count": e(1), "info": e(4)}}
    t = DTYPES[c["dtype"]]
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)  # noqa: E731
    d, hq, hk = c["head_dim"], c["q_heads"], c["kv_heads"]
    if c["kind"] == "rope":
        n, p = c["tokens"], c["page"]
        qkv = normal(n, hq + 2 * hk, d).mul_(1.5).to(t)  # what the projection writes: q, k and v heads of a token side by side
        blocks = -(-n // p) + 2
        slots = torch.randperm(blocks * p, generator=g, device="cuda")[:n].contiguous()
        if c["skip"]:
            slots[-min(c["skip"], n):] = -1  # rows behind the last token of a padded batch
        pos = torch.randint(0, c["far"], (c["axes"], n), generator=g, device="cuda", dtype=torch.int32)
        half = c["rot"] // 2
        freq = (10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)).float()
        cut = [half // c["axes"] + (1 if i < half % c["axes"] else 0) for i in range(c["axes"])]
        w = [normal(d).mul_(0.1).add_(0.0 if c["gemma"] else 1.0).to(t) if c["norm"] else None for _ in range(2)]
        return {"case": c, "q": qkv[:, :hq], "k": qkv[:, hq:hq + hk], "v": qkv[:, hq + hk:], "positions": pos, "freq": freq, "sections": cut, "wq": w[0], "wk": w[1],
                "slots": slots, "k_cache": normal(blocks, p, hk, d).to(t), "v_cache": normal(blocks, p, hk, d).to(t), "q_out": torch.empty(n, hq, d, dtype=t, device="cuda")}
    cached, new = _lens(c)
    lens = [x + n for x, n in zip(cached, new)]
    table, _, total = _pages(c, lens, g)
    rows = sum(new) + c["spare"]
    cu = np.concatenate([[0], np.cumsum(new)]).tolist()
    slopes = torch.tensor([2.0 ** (-8.0 * (i + 1) / hq) for i in range(hq)], dtype=torch.float32, device="cuda") if c["slopes"] else None
    return {"case": c, "q": normal(rows, hq, d).to(t), "k_cache": normal(total, c["page"], hk, d).to(t), "v_cache": normal(total, c["page"], hk, d).to(t),
            "table": table, "cu": _ints(cu), "lens": _ints(lens), "slopes": slopes, "prefix": _ints([min(c["prefix"], x) for x in lens]) if c["prefix"] else None,
            "max_new": max(new), "max_len": max(lens), "out": torch.zeros(rows, hq, d, dtype=t, device="cuda"),
            "lse": torch.zeros(rows, hq, dtype=torch.float32, device="cuda")}


def _plan(s):
    page, table, n = s["page"], s["table"], s["out"]["slots"].numel()
    cached, new = s["cached"].long(), s["new"].long()
    have = (cached + page - 1) // page
    need = (cached + new + page - 1) // page - have
    last = torch.cumsum(need, 0)
    first, count = last - need, s["count"].long()
    col = torch.arange(table.shape[1], device=table.device)
    j = col - have[:, None]
    pick = (count - 1 - first[:, None] - j).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where((j >= 0) & (j < need[:, None]), s["free"][pick], table))
    cu = torch.cat([torch.zeros_like(last[:1]), torch.cumsum(new, 0)])
    t = torch.arange(n, device=table.device)
    r = torch.searchsorted(cu[1:], t, right=True)
    there = r < new.numel()
    r = r.clamp(max=new.numel() - 1)
    pos = cached[r] + t - cu[r]
    slot = table[r, torch.where(there, pos // page, 0)].long() * page + pos % page
    info = torch.stack([cu[-1], last[-1], torch.zeros_like(last[-1]), last[-1]])
    i32 = lambda x: x.to(torch.int32)  # noqa: E731
    return {"table": table, "cu": i32(cu), "lens": i32(cached + new), "slots": torch.where(there, slot, -1), "positions": i32(torch.where(there, pos, 0)),
            "count": i32(count - last[-1]), "info": i32(info)}


def _axis_of(sections, dealt):
    """The position axis of each frequency: whole sections after one another, or dealt in turn until a section is full."""
    if not dealt:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    return [a for k in range(max(sections)) for a, n in enumerate(sections) if k < n]


def _rope_head(x, w, gemma, cos, sin, rot, pairs):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * (w.float() + 1.0 if gemma else w.float())
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if pairs else (r[..., :rot // 2], r[..., rot // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _rope(s):
    c, t = s["case"], s["q"].dtype
    axis = torch.tensor(_axis_of(s["sections"], c["dealt"]), device="cuda")
    angle = s["positions"].double()[axis].t() * s["freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    q = _rope_head(s["q"], s["wq"], c["gemma"], cos, sin, c["rot"], c["pairs"]).to(t)
    k = _rope_head(s["k"], s["wk"], c["gemma"], cos, sin, c["rot"], c["pairs"]).to(t)
    there = s["slots"] >= 0
    kc, vc = s["k_cache"].view(-1, *k.shape[1:]), s["v_cache"].view(-1, *k.shape[1:])
    kc[s["slots"][there]] = k[there]
    vc[s["slots"][there]] = s["v"][there]
    return q, s["k_cache"], s["v_cache"]


def _attend(s):
    c, q, page = s["case"], s["q"], s["case"]["page"]
    hk, dev = c["kv_heads"], q.device
    n, length = torch.arange(s["max_new"], device=dev), torch.arange(s["max_len"], device=dev)
    first, lens = s["cu"][:-1].long(), s["lens"].long()
    new = s["cu"][1:].long() - first
    row = (first[:, None] + n).clamp(max=q.shape[0] - 1)
    qf = q[row].float().unflatten(2, (hk, -1))                                        # [R, N, Hk, G, D]
    slot = (s["table"].clamp(min=0).long() * page)[:, length // page] + length % page  # [R, L]
    kf, vf = (x.flatten(0, 1)[slot].float() for x in (s["k_cache"], s["v_cache"]))    # [R, L, Hk, D]
    w = torch.einsum("rnhgd,rlhd->rhgnl", qf, kf).mul_(c["head_dim"] ** -0.5)
    if c["cap"]:
        w = w.div_(c["cap"]).tanh_().mul_(c["cap"])
    p = (lens - new)[:, None] + n                                                     # the queries' positions [R, N]
    far = p[:, :, None] - length                                                      # [R, N, L]
    if s["slopes"] is not None:
        w -= s["slopes"].view(hk, -1)[:, :, None, None] * far[:, None, None].abs().float()
    see = torch.ones_like(far, dtype=torch.bool)
    if c["causal"]:
        see &= far >= 0
    if c["window"]:
        see &= far < c["window"]
    if s["prefix"] is not None:
        see |= length < s["prefix"].long()[:, None, None]
    see &= (length < lens[:, None])[:, None]
    w.masked_fill_(~see[:, None, None], -math.inf)
    top = w.amax(-1, keepdim=True).clamp(min=-1e30)
    w = w.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.einsum("rhgnl,rlhd->rhgnd", w, vf) / torch.where(total > 0, total, 1.0)
    lse = top + torch.log(total)
    there = n < new[:, None]
    s["out"][row[there]] = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[there].to(q.dtype)
    s["lse"][row[there]] = lse[..., 0].permute(0, 3, 1, 2).flatten(2, 3)[there]
    return s["out"], s["lse"]


_kept = {}


def _context():
    """The program's one context on the device."""
    if "ctx" not in _kept:
        import tensor_all_reduce_gb300 as tar
        _kept["ctx"] = tar.Context(torch.cuda.current_device())
    return _kept["ctx"]


def run(s):
    c = s["case"]
    if not own:
        return {"plan": _plan, "rope": _rope, "attend": _attend}[c["kind"]](s)
    ctx = _context()
    if c["kind"] == "plan":
        o = s["out"]
        ctx.paged_plan(s["cached"], s["new"], s["free"], s["count"], s["table"], s["page"], cu_q=o["cu"], seq_lens=o["lens"], slots=o["slots"],
                       positions=o["positions"], free_count_out=o["count"], info=o["info"])
        return {"table": s["table"], **o}
    if c["kind"] == "rope":
        ctx.qk_norm_rope(s["q"], s["k"], s["v"], s["positions"], s["freq"], q_weight=s["wq"], k_weight=s["wk"], eps=1e-6, gemma=c["gemma"], pairs=c["pairs"],
                         sections=s["sections"], dealt=c["dealt"], k_cache=s["k_cache"], v_cache=s["v_cache"], slots=s["slots"], q_out=s["q_out"], want_k_out=False)
        return s["q_out"], s["k_cache"], s["v_cache"]
    ctx.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["lens"], causal=c["causal"], window=c["window"], softcap=c["cap"],
                        slopes=s["slopes"], prefix_lens=s["prefix"], out=s["out"], lse=s["lse"])
    return s["out"], s["lse"]


def _visible(c):
    """Over the requests: visible (query, key) pairs of a head, and keys that some query sees."""
    pairs, keys = 0, 0
    for cached, n in zip(*_lens(c)):
        if not n:
            continue
        length = cached + n
        p = np.arange(cached, length)
        pre = min(c["prefix"], length)
        high = np.minimum(p + 1, length) if c["causal"] else np.full(n, length)
        low = np.maximum(p - c["window"] + 1, 0) if c["window"] else np.zeros(n, dtype=np.int64)
        pairs += int((pre + np.maximum(high - np.maximum(low, pre), 0)).sum())
        keys += int(pre + max(high.max() - max(low.min(), pre), 0))
    return pairs, keys


def work(case):
    c = case
    if c["kind"] == "plan":
        cached, new = _lens(c)
        p = c["page"]
        taken = sum(-(-(x + n) // p) - -(-x // p) for x, n in zip(cached, new))
        used = sum(-(-(x + n) // p) - x // p for x, n in zip(cached, new) if n)
        return {"bytes": 4 * (4 * c["requests"] + 2 * taken + used) + 12 * (sum(new) + c["spare"]) + 32, "flops": 0}
    es, d = 2, c["head_dim"]
    if c["kind"] == "rope":
        n, heads = c["tokens"], c["q_heads"] + 2 * c["kv_heads"]
        kept = n - min(c["skip"], n)
        moved = es * d * (n * 2 * c["q_heads"] + kept * 4 * c["kv_heads"])
        return {"bytes": moved + n * (8 + 4 * c["axes"]), "flops": n * heads * d * 6}
    pairs, keys = _visible(c)
    rows = sum(_lens(c)[1])
    return {"bytes": es * d * (2 * rows * c["q_heads"] + 2 * keys * c["kv_heads"]) + 4 * rows * c["q_heads"], "flops": 4 * d * c["q_heads"] * pairs}


def _exact_plan(s, c):
    page, cached, new = c["page"], s["cached"].tolist(), s["new"].tolist()
    table, free = s["table"].cpu().numpy().copy(), s["free"].tolist()
    slots, positions, cu, lens = [], [], [0], []
    taken = 0
    for r, (x, n) in enumerate(zip(cached, new)):
        for j in range(-(-x // page), -(-(x + n) // page)):
            table[r, j] = free.pop()
            taken += 1
        for i in range(x, x + n):
            positions.append(i)
            slots.append(int(table[r, i // page]) * page + i % page)
        cu.append(cu[-1] + n)
        lens.append(x + n)
    more = s["out"]["slots"].numel() - len(slots)
    a = lambda v: np.array(v, dtype=np.int32)  # noqa: E731
    return {"table": table, "cu": a(cu), "lens": a(lens), "slots": np.array(slots + [-1] * more, dtype=np.int64), "positions": a(positions + [0] * more),
            "count": a([len(free)]), "info": a([len(slots), taken, 0, taken])}


def _exact_rope(s, c):
    out = []
    axis = _axis_of(s["sections"], c["dealt"])
    turn = torch.stack([s["positions"][a].double() * s["freq"][i].double() for i, a in enumerate(axis)], -1)
    unit = torch.polar(torch.ones_like(turn), turn)[:, None]  # a pair is a complex number, turned by the angle
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt((y.square().sum(-1, keepdim=True) / c["head_dim"]) + 1e-6) * (w.double() + (1.0 if c["gemma"] else 0.0))
        y = y.clone()
        half = c["rot"] // 2
        i = torch.arange(half, device="cuda")
        re, im = (2 * i, 2 * i + 1) if c["pairs"] else (i, i + half)
        z = torch.complex(y[..., re], y[..., im]) * unit
        y[..., re], y[..., im] = z.real, z.imag
        out.append(y)
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    at = s["slots"].clamp(min=0)
    for cache, rows in ((kc, out[1]), (vc, s["v"].double())):
        keep = (s["slots"] >= 0).nonzero()[:, 0]
        cache[at[keep] // c["page"], at[keep] % c["page"]] = rows[keep]
    return out[0], kc, vc


def _exact_attend(s, c):
    out, lse = s["out"].double(), s["lse"].double()
    cu, lens, g = s["cu"].tolist(), s["lens"].tolist(), c["q_heads"] // c["kv_heads"]
    for r in range(c["requests"]):
        n, length = cu[r + 1] - cu[r], lens[r]
        if n == 0:
            continue
        pages = s["table"][r, : -(-length // c["page"])].long()
        i = torch.arange(length - n, length, device="cuda")[:, None]
        j = torch.arange(length, device="cuda")[None]
        hidden = torch.zeros(n, length, dtype=torch.bool, device="cuda")
        if c["causal"]:
            hidden |= j > i
        if c["window"]:
            hidden |= j <= i - c["window"]
        if s["prefix"] is not None:
            hidden &= j >= s["prefix"][r]
        for h in range(c["kv_heads"]):
            k, v = (x[pages, :, h].double().flatten(0, 1)[:length] for x in (s["k_cache"], s["v_cache"]))
            for e in range(h * g, h * g + g):
                z = s["q"][cu[r]:cu[r + 1], e].double() @ k.t() / math.sqrt(c["head_dim"])
                if c["cap"]:
                    z = c["cap"] * torch.tanh(z / c["cap"])
                if s["slopes"] is not None:
                    z = z - s["slopes"][e].double() * (i - j).abs()
                z = z.masked_fill(hidden, -math.inf)
                lse[cu[r]:cu[r + 1], e] = torch.logsumexp(z, -1)
                out[cu[r]:cu[r + 1], e] = torch.nan_to_num(torch.softmax(z, -1)) @ v
    return out, lse


def exact(case, seed):
    c = case
    if c["kind"] == "attend" and 4.0 * c["head_dim"] * c["q_heads"] * _visible(c)[0] > 8e12:
        return None
    return {"plan": _exact_plan, "rope": _exact_rope, "attend": _exact_attend}[c["kind"]](prepare(c, seed), c)
