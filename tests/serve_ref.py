"""Plain 64-bit forms of the attention block's operators and their error bounds, for the tests."""
import math

import torch

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def half_step(dt):
    """Largest relative error of one rounding to nearest."""
    return torch.finfo(dt).eps / 2


def smallest(dt):
    """Half the spacing of the subnormal values."""
    return torch.finfo(dt).tiny * torch.finfo(dt).eps / 2


def plan(cached, new, free, page, table, max_tokens):
    """The plan as lists; table (a list of lists) is changed in place."""
    need = [-(-(c + n) // page) - -(-c // page) for c, n in zip(cached, new)]
    code = 0
    if sum(need) > len(free):
        code = 1
    if any(-(-(c + n) // page) > len(t) for c, n, t in zip(cached, new, table)):
        code = 2
    if sum(new) > max_tokens:
        code = 3
    if code:
        return {"cu_q": [0] * (len(new) + 1), "seq_lens": list(cached), "slots": [-1] * max_tokens, "positions": [0] * max_tokens,
                "free_count": [len(free)], "info": [0, 0, code, sum(need)]}
    free, slots, positions, cu = list(free), [], [], [0]
    for c, n, t in zip(cached, new, table):
        for j in range(-(-c // page), -(-(c + n) // page)):
            t[j] = free.pop()
        for pos in range(c, c + n):
            slots.append(t[pos // page] * page + pos % page)
            positions.append(pos)
        cu.append(cu[-1] + n)
    pad = max_tokens - len(slots)
    return {"cu_q": cu, "seq_lens": [c + n for c, n in zip(cached, new)], "slots": slots + [-1] * pad, "positions": positions + [0] * pad,
            "free_count": [len(free)], "info": [len(slots), sum(need), 0, sum(need)]}


def axis_of(sections, dealt):
    if not dealt:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    return [a for k in range(max(sections)) for a, n in enumerate(sections) if k < n]


def rope(x, weight, eps, gemma, positions, inv_freq, pairs, axis):
    """(exact values, bound on the kernel's error) of heads x [T, H, D]; positions [A, T]; CPU tensors.

    The bound: one rounding to the type, and in fp32 the norm (a sum of D squares by at most D / 32 + 5
    additions in a row, its root and two products: under 16 roundings of 2^-24 for D <= 256), sine and
    cosine (the turn cut to 24 bits: pi 2^-25; sincospi to 2 ulp: 2^-23), and three roundings of the
    rotation: under 32 of 2^-24, relative to |a| + |b|."""
    y = x.double()
    if weight is not None:
        w = weight.double() + (1.0 if gemma else 0.0)
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * w
    out, size = y.clone(), y.abs()
    half = 0 if inv_freq is None else inv_freq.numel()
    if half:
        theta = torch.stack([positions[a].double() * inv_freq[i].double() for i, a in enumerate(axis)], -1)[:, None]
        i = torch.arange(half)
        ia, ib = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        a, b = y[..., ia], y[..., ib]
        out[..., ia] = a * theta.cos() - b * theta.sin()
        out[..., ib] = b * theta.cos() + a * theta.sin()
        size[..., ia] = size[..., ib] = a.abs() + b.abs()
    if weight is None and not half:
        return out, torch.zeros_like(out)
    fp32 = 2.0 ** -19 * size
    return out, half_step(x.dtype) * (out.abs() + fp32) + fp32 + smallest(x.dtype)


def attention(q, k_cache, v_cache, table, cu, lens, scale, causal=True, window=0, softcap=0.0, slopes=None, prefix=None):
    """(out, lse, bound of out, bound of lse), CPU float64; rows of no request are NaN.

    The bounds, with u the half step of the type, N keys, D the head size: a score is a sum of D products in
    fp32, then scaled, bent and turned to log2 units: |ds| <= (2 D + 16) 2^-24 (sum |q k| scale + cap +
    bias); a weight is exp of a difference of two scores, off by 2 |ds| + 2^-21 relative, then rounded to the type: u
    relative, or half a subnormal step for weights of 2^8 at most relative to the largest; the sums of N terms add N 2^-23."""
    t, hq, d = q.shape
    page, hk = k_cache.shape[1], k_cache.shape[2]
    g, u, dt = hq // hk, half_step(q.dtype), q.dtype
    out = torch.full((t, hq, d), math.nan, dtype=torch.float64)
    lse = torch.full((t, hq), math.nan, dtype=torch.float64)
    eo, el = out.clone(), lse.clone()
    for r in range(len(lens)):
        lo, hi, length = cu[r], cu[r + 1], lens[r]
        n = hi - lo
        if n == 0:
            continue
        rows = torch.arange(length)
        blocks = torch.tensor([table[r][j] for j in range(-(-length // page))], dtype=torch.long)
        blocks = blocks.clamp(0, k_cache.shape[0] - 1)  # blocks that no row sees may have any number
        k = k_cache[blocks].flatten(0, 1)[:length].double()
        v = v_cache[blocks].flatten(0, 1)[:length].double()
        pos = torch.arange(length - n, length)[:, None]
        see = torch.ones(n, length, dtype=torch.bool)
        if causal:
            see &= rows <= pos
        if window:
            see &= rows > pos - window
        if prefix is not None:
            see |= rows < prefix[r]
        for h in range(hq):
            qh, kh, vh = q[lo:hi, h].double(), k[:, h // g], v[:, h // g]
            kh = torch.where(see.any(0)[:, None], kh, 0.0)  # a key that no row sees may hold anything
            s = qh @ kh.t() * scale
            size = (qh.abs() @ kh.abs().t()) * abs(scale)
            if softcap:
                s = softcap * torch.tanh(s / softcap)
                size = size + softcap
            if slopes is not None:
                bias = float(slopes[h]) * (pos - rows).abs()
                s = s - bias
                size = size + abs(bias)
            s = s.masked_fill(~see, -math.inf)
            top = s.amax(-1, keepdim=True) if length else torch.full((n, 1), -math.inf, dtype=torch.float64)
            some = top > -math.inf
            w = torch.exp(s - torch.where(some, top, 0.0))
            w = torch.where(see, w, 0.0)
            z = w.sum(-1, keepdim=True)
            p = w / torch.where(some, z, 1.0)
            o = p @ vh
            log = torch.where(some, top + torch.log(torch.where(some, z, 1.0)), -math.inf)[:, 0]
            ds = ((2 * d + 16) * 2.0 ** -24 * torch.where(see, size, 0.0).amax(-1, keepdim=True)) if length else torch.zeros(n, 1, dtype=torch.float64)
            rel = 4 * ds + 2.0 ** -20 + length * 2.0 ** -22
            spread = p @ vh.abs()
            sub = smallest(dt) * vh.abs().sum(0)
            out[lo:hi, h], lse[lo:hi, h] = o, log
            eo[lo:hi, h] = u * o.abs() + (1 + u) * ((u + rel) * spread + sub) + smallest(dt)
            el[lo:hi, h] = (2 * ds[:, 0] + 2.0 ** -20 + length * 2.0 ** -22 + 2.0 ** -22 * torch.where(some[:, 0], log.abs(), 0.0))
    return out, lse, eo, el
