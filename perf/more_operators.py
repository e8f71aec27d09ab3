"""The operators of a paged cache held in 8 bits, as a user's program calls them.

Two operators of one serving step: the append (norm and rotation of the new keys, and the write of keys and values as E4M3
codes with one scale for each block of tokens and head), and the attention of the new tokens over such a cache.  `run`
computes them in plain torch operations, or through the framework where `own` is true; `exact` is the definition in 64
bits."""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn
LOW, HIGH = 2.0 ** -32, 2.0 ** 32  # the range of the scales


def listed():
    return [
        # decode of 16 requests (the benchmark's decode rows) on one of four ranks: 2 key heads of 128
        {"name": "append decode 16", "kind": "append", "dtype": "bf16", "kv_heads": 2, "head_dim": 128, "page": 16, "requests": 16, "new": 1, "ctx": 2000,
         "mode": "ragged", "rot": 128, "pairs": False, "axes": 1, "dealt": False, "norm": True, "gemma": False, "far": 0, "spare": 0, "lengths": 1},
        # decode of a full batch with all key heads, keys rotated without a norm, padded for a captured graph
        {"name": "append decode 256", "kind": "append", "dtype": "fp16", "kv_heads": 8, "head_dim": 64, "page": 32, "requests": 256, "new": 1, "ctx": 600,
         "mode": "ragged", "rot": 64, "pairs": False, "axes": 1, "dealt": False, "norm": False, "gemma": False, "far": 0, "spare": 6, "lengths": 2},
        # a scheduler's step: chunks that begin inside a block together with single tokens (about the benchmark's 2800 rows), half of each head rotated, gemma weights
        {"name": "append mixed 2800", "kind": "append", "dtype": "bf16", "kv_heads": 8, "head_dim": 128, "page": 16, "requests": 64, "new": 690, "ctx": 1000,
         "mode": "mixed", "rot": 64, "pairs": False, "axes": 1, "dealt": False, "norm": True, "gemma": True, "far": 0, "spare": 0, "lengths": 3},
        # image and video tokens with three position axes dealt in turn, adjacent pairs, 80-wide heads, large blocks
        {"name": "append video 16384", "kind": "append", "dtype": "fp16", "kv_heads": 16, "head_dim": 80, "page": 64, "requests": 4, "new": 4096, "ctx": 0,
         "mode": "each", "rot": 80, "pairs": True, "axes": 3, "dealt": True, "norm": True, "gemma": False, "far": 2000, "spare": 0, "lengths": 4},
        # a 4096-row chunk (the benchmark's largest) of one long prompt
        {"name": "append chunk 4096", "kind": "append", "dtype": "bf16", "kv_heads": 8, "head_dim": 128, "page": 64, "requests": 1, "new": 4096, "ctx": 4000,
         "mode": "each", "rot": 128, "pairs": False, "axes": 1, "dealt": False, "norm": True, "gemma": False, "far": 0, "spare": 0, "lengths": 5},
        # one request answers alone: latency
        {"name": "attend one token", "kind": "attend", "dtype": "bf16", "q_heads": 12, "kv_heads": 2, "head_dim": 128, "page": 16, "requests": 1,
         "new": 1, "ctx": 700, "mode": "each", "causal": True, "window": 0, "cap": 0.0, "slopes": False, "prefix": 0, "spare": 0, "even": True, "lengths": 6},
        # decode of a full batch with ragged long contexts: bound by reading the cache
        {"name": "attend decode 64", "kind": "attend", "dtype": "bf16", "q_heads": 48, "kv_heads": 8, "head_dim": 128, "page": 16, "requests": 64,
         "new": 1, "ctx": 9000, "mode": "ragged", "causal": True, "window": 0, "cap": 0.0, "slopes": False, "prefix": 0, "spare": 3, "even": True, "lengths": 7},
        # chunks together with single tokens, scores capped, sliding window, fp16, heads of 64
        {"name": "attend mixed window", "kind": "attend", "dtype": "fp16", "q_heads": 16, "kv_heads": 4, "head_dim": 64, "page": 32, "requests": 17,
         "new": 700, "ctx": 5000, "mode": "mixed", "causal": True, "window": 1024, "cap": 30.0, "slopes": False, "prefix": 0, "spare": 0, "even": True, "lengths": 8},
        # prompts with a prefix that sees itself both ways and a bias by distance, 96-wide heads, scales that are no powers of two
        {"name": "attend prefix bias", "kind": "attend", "dtype": "bf16", "q_heads": 8, "kv_heads": 8, "head_dim": 96, "page": 64, "requests": 6,
         "new": 1500, "ctx": 0, "mode": "ragged", "causal": True, "window": 0, "cap": 0.0, "slopes": True, "prefix": 256, "spare": 0, "even": False, "lengths": 9},
        # one key head of 256, a chunk over a middle context
        {"name": "attend wide heads", "kind": "attend", "dtype": "bf16", "q_heads": 8, "kv_heads": 1, "head_dim": 256, "page": 16, "requests": 2,
         "new": 1024, "ctx": 8000, "mode": "each", "causal": True, "window": 0, "cap": 0.0, "slopes": False, "prefix": 0, "spare": 0, "even": True, "lengths": 10},
        # a 4096-row chunk of a long document: bound by the products
        {"name": "attend chunk 4096", "kind": "attend", "dtype": "bf16", "q_heads": 12, "kv_heads": 2, "head_dim": 128, "page": 64, "requests": 1,
         "new": 4096, "ctx": 28000, "mode": "each", "causal": True, "window": 0, "cap": 0.0, "slopes": False, "prefix": 0, "spare": 0, "even": True, "lengths": 11},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    lengths, dtype, mode = rng.randrange(1, 1 << 20), rng.choice(["bf16", "fp16"]), rng.choice(["ragged", "mixed", "each"])
    if rng.random() < 0.4:
        kv_heads, head_dim = rng.choice([1, 2, 4, 7, 8, 16]), rng.choice([64, 80, 96, 128, 128, 256])
        axes, rot = rng.choice([1, 1, 2, 3, 4]), rng.choice([head_dim, head_dim, head_dim // 2, 2 * (head_dim // 8)])
        most = min(16384, 16384 * 16 * 80 // (kv_heads * head_dim))
        requests = _log(rng, 1, 300)
        new = rng.choice([1, 1, 3, _log(rng, 1, max(1, most // requests))])
        ctx = rng.choice([0, _log(rng, 1, 4000)])
        while requests * (ctx + new) * kv_heads * head_dim > 3e8:
            ctx = ctx * 3 // 4
        return {"kind": "append", "dtype": dtype, "kv_heads": kv_heads, "head_dim": head_dim, "page": rng.choice([8, 16, 16, 24, 32, 64, 128]),
                "requests": requests, "new": new, "ctx": ctx, "mode": mode, "rot": rot, "pairs": rng.random() < 0.4, "axes": axes,
                "dealt": axes > 1 and rng.random() < 0.5, "norm": rng.random() < 0.7, "gemma": rng.random() < 0.3,
                "far": _log(rng, 100, 1000000) if axes > 1 else 0, "spare": rng.choice([0, 0, 3]), "lengths": lengths}
    q_heads, kv_heads = rng.choice([(12, 2), (6, 1), (48, 8), (8, 8), (16, 4), (8, 1), (16, 16), (20, 4), (7, 1)])
    head_dim, requests = rng.choice([64, 80, 96, 128, 128, 128, 256]), _log(rng, 1, 64)
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
            "spare": rng.choice([0, 0, 5]), "even": rng.random() < 0.7, "lengths": lengths}


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


def _pages(c, g):
    """A shuffled pool of blocks, and each request's table row as far as its tokens of this step go."""
    p = c["page"]
    need = [-(-(x + n) // p) for x, n in zip(*_lens(c))]
    total = sum(need) + 8 + sum(need) // 16
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    width = max(max(need), 1) + 3
    col = torch.arange(width, device="cuda")
    h = torch.tensor(need, device="cuda")
    place = ((torch.cumsum(h, 0) - h)[:, None] + col).clamp(max=total - 1)
    return torch.where(col < h[:, None], order[place], -1).contiguous(), total


def _cache(blocks, page, heads, dim, even, g):
    """Codes and scales of a cache of normal values whose size differs from block to block and head to head."""
    x = torch.randn((blocks, page, heads, dim), generator=g, device="cuda", dtype=torch.float16)
    size = torch.exp2(torch.randint(-4, 3, (blocks, heads), generator=g, device="cuda").float() / 2)
    scale = x.abs().amax((1, 3)).float() * size / 448
    if even:
        scale = torch.exp2(torch.ceil(torch.log2(scale)))
    return x.mul_((size / scale).half()[:, None, :, None]).clamp_(-448, 448).to(E4M3), scale


def prepare(case, seed):
    c, g = case, _gen(seed)
    t, d, hk = DTYPES[c["dtype"]], c["head_dim"], c["kv_heads"]
    normal = lambda *shape: torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)  # noqa: E731
    cached, new = _lens(c)
    lens, rows = [x + n for x, n in zip(cached, new)], sum(new) + c["spare"]
    table, total = _pages(c, g)
    s = {"case": c, "table": table, "cu": _ints(np.concatenate([[0], np.cumsum(new)]).tolist()), "lens": _ints(lens)}
    s["kc"], s["ks"] = _cache(total, c["page"], hk, d, c.get("even", True), g)
    s["vc"], s["vs"] = _cache(total, c["page"], hk, d, c.get("even", True), g)
    if c["kind"] == "append":
        kv = normal(rows, 2 * hk, d).mul_(1.5).to(t)  # what the projection writes: k and v heads of a token side by side
        s["k"], s["v"] = kv[:, :hk], kv[:, hk:]
        half = c["rot"] // 2
        s["freq"] = (10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)).float()
        s["sections"] = [half // c["axes"] + (1 if i < half % c["axes"] else 0) for i in range(c["axes"])]
        s["w"] = normal(d).mul_(0.1).add_(0.0 if c["gemma"] else 1.0).to(t) if c["norm"] else None
        place = [x + i for x, n in zip(cached, new) for i in range(n)] + [0] * c["spare"]
        s["positions"] = torch.randint(0, c["far"], (c["axes"], rows), generator=g, device="cuda", dtype=torch.int32) if c["axes"] > 1 else _ints(place)[None]
        return s
    hq = c["q_heads"]
    s["q"] = normal(rows, hq, d).to(t)
    s["slopes"] = torch.tensor([2.0 ** (-8.0 * (i + 1) / hq) for i in range(hq)], dtype=torch.float32, device="cuda") if c["slopes"] else None
    s["prefix"] = _ints([min(c["prefix"], x) for x in lens]) if c["prefix"] else None
    s["max_new"], s["max_len"] = max(new), max(lens)
    s["out"] = torch.zeros(rows, hq, d, dtype=t, device="cuda")
    s["lse"] = torch.zeros(rows, hq, dtype=torch.float32, device="cuda")
    return s


def _axis_of(sections, dealt):
    """The position axis of each frequency: whole sections after one another, or dealt in turn until a section is full."""
    if not dealt:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    return [a for k in range(max(sections)) for a, n in enumerate(sections) if k < n]


def _turned(s):
    """The new keys after norm and rotation, in 32 bits (angles in 64)."""
    c, rot = s["case"], s["case"]["rot"]
    x = s["k"].float()
    if s["w"] is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * (s["w"].float() + 1.0 if c["gemma"] else s["w"].float())
    axis = torch.tensor(_axis_of(s["sections"], c["dealt"]), device="cuda")
    angle = s["positions"].double()[axis].t() * s["freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if c["pairs"] else (r[..., :rot // 2], r[..., rot // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([a, b], -1).flatten(-2) if c["pairs"] else torch.cat([a, b], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _append(s):
    page, codes = s["case"]["page"], (s["kc"].view(torch.uint8), s["vc"].view(torch.uint8))
    first, lens = s["cu"][:-1].long(), s["lens"].long()
    new = s["cu"][1:].long() - first
    t = torch.arange(s["k"].shape[0], device="cuda")
    r = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    there = r < new.numel()
    t, r = t[there], r[there]
    place = (lens - new)[r] + t - first[r]
    block, off = s["table"][r, place // page].long(), place % page
    held = torch.zeros(s["ks"].shape[0], dtype=torch.long, device="cuda")  # tokens that a block held before
    held[block] = ((lens - new)[r] - place // page * page).clamp(min=0)
    touched = torch.zeros_like(held, dtype=torch.bool)
    touched[block] = True
    was = torch.arange(page, device="cuda") < held[:, None]
    for x, cache, scale in ((_turned(s)[t], codes[0], s["ks"]), (s["v"][t].float(), codes[1], s["vs"])):
        top = torch.zeros_like(scale).index_reduce_(0, block, x.abs().amax(-1), "amax")
        m, e = torch.frexp(top)
        fresh = torch.ldexp(torch.ones_like(top), e - 9 + (m > 0.875)).clamp(LOW, HIGH)  # 448 = 0.875 * 2^9
        fresh = torch.where(top > 0, fresh, LOW)
        now = torch.where((held > 0)[:, None], torch.maximum(scale, fresh), fresh)
        again = cache.view(E4M3).float() * (scale / now)[:, None, :, None]
        cache.copy_(torch.where((was & touched[:, None])[:, :, None, None], again.to(E4M3).view(torch.uint8), cache))
        cache[block, off] = (x / now[block][..., None]).to(E4M3).view(torch.uint8)
        scale.copy_(torch.where(touched[:, None], now, scale))
    return s["kc"], s["vc"], s["ks"], s["vs"]


def _attend(s):
    c, q, page = s["case"], s["q"], s["case"]["page"]
    hk, dev = c["kv_heads"], q.device
    n, length = torch.arange(s["max_new"], device=dev), torch.arange(s["max_len"], device=dev)
    first, lens = s["cu"][:-1].long(), s["lens"].long()
    new = s["cu"][1:].long() - first
    row = (first[:, None] + n).clamp(max=q.shape[0] - 1)
    qf = q[row].float().unflatten(2, (hk, -1))                                # [R, N, Hk, G, D]
    block = s["table"].clamp(min=0).long()[:, length // page]                 # [R, L]
    slot = block * page + length % page
    kf, vf = (x.view(torch.uint8).flatten(0, 1)[slot].view(E4M3).float().mul_(y[block][..., None])
              for x, y in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))           # [R, L, Hk, D]
    w = torch.einsum("rnhgd,rlhd->rhgnl", qf, kf).mul_(c["head_dim"] ** -0.5)
    if c["cap"]:
        w = w.div_(c["cap"]).tanh_().mul_(c["cap"])
    p = (lens - new)[:, None] + n                                             # the queries' positions [R, N]
    far = p[:, :, None] - length                                              # [R, N, L]
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
        return {"append": _append, "attend": _attend}[c["kind"]](s)
    ctx = _context()
    if c["kind"] == "append":
        ctx.paged_append_fp8(s["k"], s["v"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["cu"], s["lens"], positions=s["positions"], inv_freq=s["freq"],
                             k_weight=s["w"], eps=1e-6, gemma=c["gemma"], pairs=c["pairs"], sections=s["sections"], dealt=c["dealt"])
        return s["kc"], s["vc"], s["ks"], s["vs"]
    ctx.paged_attention_fp8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["cu"], s["lens"], causal=c["causal"], window=c["window"],
                            softcap=c["cap"], slopes=s["slopes"], prefix_lens=s["prefix"], out=s["out"], lse=s["lse"])
    return s["out"], s["lse"]


def _visible(c):
    """Over the requests: visible (query, key) pairs of a head, keys that some query sees, and their blocks."""
    pairs, keys, blocks = 0, 0, 0
    for cached, n in zip(*_lens(c)):
        if not n:
            continue
        length = cached + n
        p = np.arange(cached, length)
        pre = min(c["prefix"], length)
        high = np.minimum(p + 1, length) if c["causal"] else np.full(n, length)
        low = np.maximum(p - c["window"] + 1, 0) if c["window"] else np.zeros(n, dtype=np.int64)
        pairs += int((pre + np.maximum(high - np.maximum(low, pre), 0)).sum())
        seen = int(pre + max(high.max() - max(low.min(), pre), 0))
        keys += seen
        blocks += -(-seen // c["page"])
    return pairs, keys, blocks


def work(case):
    c, d, hk = case, case["head_dim"], case["kv_heads"]
    cached, new = _lens(c)
    rows = sum(new)
    if c["kind"] == "append":  # keys and values once in 16 bits and once in 8, a scale read where a block held tokens, written for each that is touched
        page = c["page"]
        touched = sum(-(-(x + n) // page) - x // page for x, n in zip(cached, new) if n)
        held = sum(1 for x, n in zip(cached, new) if n and x % page)
        return {"bytes": 6 * rows * hk * d + 8 * hk * (touched + held) + 4 * rows * c["axes"] + 4 * touched, "flops": rows * hk * d * 9}
    pairs, keys, blocks = _visible(c)
    return {"bytes": 4 * rows * c["q_heads"] * d + 2 * keys * hk * d + 8 * blocks * hk + 4 * rows * c["q_heads"], "flops": 4 * d * c["q_heads"] * pairs}


def _round_e4m3(x):
    """To the nearest E4M3 value, ties to the even one: three fraction bits, exponents from -6 on."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), (e - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _exact_append(s, c):
    page, half, table, cu, lens = c["page"], c["rot"] // 2, s["table"].tolist(), s["cu"].tolist(), s["lens"].tolist()
    k = s["k"].double()
    if s["w"] is not None:
        k = k / torch.sqrt((k.square().sum(-1, keepdim=True) / c["head_dim"]) + 1e-6) * (s["w"].double() + (1.0 if c["gemma"] else 0.0))
    turn = torch.stack([s["positions"][a].double() * s["freq"][i].double() for i, a in enumerate(_axis_of(s["sections"], c["dealt"]))], -1)
    unit = torch.polar(torch.ones_like(turn), turn)[:, None]  # a pair is a complex number, turned by the angle
    i = torch.arange(half, device="cuda")
    re, im = (2 * i, 2 * i + 1) if c["pairs"] else (i, i + half)
    z = torch.complex(k[..., re], k[..., im]) * unit
    k = k.clone()
    k[..., re], k[..., im] = z.real, z.imag
    out = []
    for rows, cache, scale in ((k, s["kc"], s["ks"]), (s["v"].double(), s["vc"], s["vs"])):
        cache, scale = cache.double(), scale.double()
        for r, length in enumerate(lens):
            start = length - (cu[r + 1] - cu[r])
            at = start
            while at < length:  # one block after another
                b, low = table[r][at // page], at // page * page
                end = min(low + page, length)
                x = rows[cu[r] + at - start:cu[r] + end - start]
                top = x.abs().amax((0, 2))
                need = torch.exp2(torch.ceil(torch.log2(top / 448)))
                need = torch.where(need / 2 * 448 >= top, need / 2, need).clamp(LOW, HIGH)  # a logarithm may come out above a whole number
                if at > low:
                    need = torch.maximum(need, scale[b])
                    cache[b, :at - low] = _round_e4m3(cache[b, :at - low] * (scale[b] / need)[None, :, None])
                cache[b, at - low:end - low] = _round_e4m3(x / need[None, :, None])
                scale[b] = need
                at = end
        out += [cache, scale]
    return out[0], out[2], out[1], out[3]


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
            k, v = ((x.view(torch.uint8)[pages, :, h].view(E4M3).double() * y[pages, h].double()[:, None, None]).flatten(0, 1)[:length]
                    for x, y in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
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
    return {"append": _exact_append, "attend": _exact_attend}[c["kind"]](prepare(c, seed), c)
