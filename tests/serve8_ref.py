"""Plain 64-bit forms of the operators over a cache held in 8 bits and their error bounds, for the tests."""
import math

import torch

import serve_ref as ref

E4M3 = torch.float8_e4m3fn
LOW, HIGH = 2.0 ** -32, 2.0 ** 32


def spacing(x):
    """Distance of neighbouring E4M3 values at x (three fraction bits, exponents from -6 on)."""
    _, e = torch.frexp(x.double())
    return torch.ldexp(torch.ones_like(x, dtype=torch.float64), (e - 1).clamp(min=-6) - 3)


def round_e4m3(x):
    """To nearest, ties to even, saturating; CPU float64."""
    s = spacing(x)
    return (torch.round(x / s) * s).clamp(-448.0, 448.0)


def fresh(top):
    """The smallest power of two 2^e with top <= 448 * 2^e, cut to the scales' range."""
    if top == 0:
        return LOW
    e = math.frexp(top)[1] - 10
    while 448.0 * 2.0 ** e < top:
        e += 1
    return min(max(2.0 ** e, LOW), HIGH)


def values(cache, scale):
    """What a cache [blocks, page, heads, dim] of codes stands for."""
    return cache.view(E4M3).double() * scale.double()[:, None, :, None]


def check_append(before, after, k, v, ek, ev, table, cu, lens, page):
    """A cache after an append, against the definition; k and v are the rows as they are to be stored (float64)
    and ek, ev the bounds on their errors before the rounding to codes.  `before`, `after`: (k codes, v codes, k
    scales, v scales), CPU, codes as uint8."""
    blocks, _, heads, _ = before[0].shape
    touched = {}
    for r, length in enumerate(lens):
        n = cu[r + 1] - cu[r]
        for i in range(n):
            at = length - n + i
            b = table[r][at // page]
            touched.setdefault(b, (max(length - n - at // page * page, 0), []))[1].append((at % page, cu[r] + i))
    for y, e, which in ((k, ek, 0), (v, ev, 1)):
        old, new, so, sn = before[which], after[which], before[which + 2], after[which + 2]
        rest = torch.ones(blocks, dtype=torch.bool)
        rest[list(touched)] = False
        assert torch.equal(old[rest], new[rest]) and torch.equal(so[rest], sn[rest])
        for b, (held, rows) in touched.items():
            places, at = [p for p, _ in rows], [t for _, t in rows]
            x, err = y[at], e[at]
            same = torch.ones(old.shape[1], dtype=torch.bool)
            same[places] = False
            same[:held] = False
            assert torch.equal(old[b][same], new[b][same])  # behind the last token
            for h in range(heads):
                a, z = x[:, h].abs(), err[:, h]
                some = torch.isfinite(a)
                a, z = torch.where(some, a, 0.0), torch.where(some, z, 0.0)
                was = min(max(float(so[b, h]), LOW), HIGH) if held else LOW
                low, high = (max(was, fresh(float(t))) for t in ((a - z).amax(), (a + z).amax()))
                s = float(sn[b, h])
                assert s in (low, high), (b, h, s, low, high)
                if held:
                    c = old[b, :held, h].view(E4M3).double()
                    want = c if s == was else round_e4m3(c * was / s)
                    got = new[b, :held, h].view(E4M3).double()
                    assert torch.equal(got.isnan(), c.isnan()) and torch.equal(got.nan_to_num(0.0), want.nan_to_num(0.0))
                c = new[b, places, h].view(E4M3).double()
                assert torch.equal(c.isnan(), ~some[:, :])
                t, d = torch.where(some, x[:, h], 0.0) / s, z / s
                over = (c.nan_to_num(0.0) - t.clamp(-448.0, 448.0)).abs() - (spacing(t.abs() + d) / 2 + d)
                assert (over <= 0).all(), (b, h, over.max())
                if not d.any():
                    assert torch.equal(c.nan_to_num(0.0), round_e4m3(t))


def turned(k, weight, eps, gemma, positions, freq, pairs, axis):
    """(k after norm and rotation, bound on its error in fp32): serve_ref's form without the rounding to 16 bits,
    whose bound is half a step of the type and an fp32 part; here the latter alone."""
    want, _ = ref.rope(k, weight, eps, gemma, positions, freq, pairs, axis)
    if weight is None and (freq is None or not freq.numel()):
        return want, torch.zeros_like(want)
    y = k.double()
    if weight is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * (weight.double() + (1.0 if gemma else 0.0))
    size, half = y.abs(), 0 if freq is None else freq.numel()
    if half:
        i = torch.arange(half)
        ia, ib = (2 * i, 2 * i + 1) if pairs else (i, i + half)
        size[..., ia] = size[..., ib] = y[..., ia].abs() + y[..., ib].abs()
    return want, 2.0 ** -19 * size


def attention(q, kc, vc, ks, vs, table, cu, lens, scale, causal=True, window=0, softcap=0.0, slopes=None, prefix=None):
    """(out, lse, bound of out, bound of lse), CPU float64; rows of no request are NaN.

    The bounds are serve_ref.attention's, for the values that the codes stand for, and two terms more.  A row of q
    is split into parts of 8 bits scaled by its largest element m: off by at most 2^-24 m an element, so a score by
    2^-24 m sum |k| scale.  A weight is held times its v scale, relative to the row's largest such product: at most
    u relative (half a step of the type), or 2^-22 of that largest product where it is small."""
    t, hq, d = q.shape
    page, hk = kc.shape[1], kc.shape[2]
    g, u, dt = hq // hk, ref.half_step(q.dtype), q.dtype
    out = torch.full((t, hq, d), math.nan, dtype=torch.float64)
    lse = torch.full((t, hq), math.nan, dtype=torch.float64)
    eo, el = out.clone(), lse.clone()
    ks, vs = (s.double().nan_to_num(LOW).clamp(LOW, HIGH) for s in (ks, vs))
    for r in range(len(lens)):
        lo, hi, length = cu[r], cu[r + 1], lens[r]
        n = hi - lo
        if n == 0:
            continue
        rows = torch.arange(length)
        blocks = torch.tensor([table[r][j] for j in range(-(-length // page))], dtype=torch.long)
        blocks = blocks.clamp(0, kc.shape[0] - 1)  # blocks that no row sees may have any number
        pick = lambda c: c.view(torch.uint8)[blocks].view(E4M3).double().flatten(0, 1)[:length]  # noqa: E731
        each = lambda s: s[blocks].repeat_interleave(page, 0)[:length]  # noqa: E731
        ck, cv, sk, sv = pick(kc), pick(vc), each(ks), each(vs)
        pos = torch.arange(length - n, length)[:, None]
        see = torch.ones(n, length, dtype=torch.bool)
        if causal:
            see &= rows <= pos
        if window:
            see &= rows > pos - window
        if prefix is not None:
            see |= rows < prefix[r]
        seen = see.any(0)[:, None]
        for h in range(hq):
            qh, s8 = q[lo:hi, h].double(), sv[:, h // g]
            kh = torch.where(seen, ck[:, h // g] * sk[:, h // g, None], 0.0)  # a key that no row sees may hold anything
            vh = torch.where(seen, cv[:, h // g] * s8[:, None], 0.0)
            s = qh @ kh.t() * scale
            size = (qh.abs() @ kh.abs().t()) * abs(scale)
            split = 2.0 ** -24 * qh.abs().amax(-1, keepdim=True) * kh.abs().sum(-1) * abs(scale)
            if softcap:
                s = softcap * torch.tanh(s / softcap)
                size = size + softcap
            if slopes is not None:
                bias = float(slopes[h]) * (pos - rows).abs()
                s = s - bias
                size = size + abs(bias)
            # t = log2(vs) is added to a score in log2 units, and taken off again: both sums are rounded
            size = size + s8.log2().abs()
            s = s.masked_fill(~see, -math.inf)
            top = s.amax(-1, keepdim=True) if length else torch.full((n, 1), -math.inf, dtype=torch.float64)
            some = top > -math.inf
            w = torch.exp(s - torch.where(some, top, 0.0))
            w = torch.where(see, w, 0.0)
            z = w.sum(-1, keepdim=True)
            p = w / torch.where(some, z, 1.0)
            o = p @ vh
            log = torch.where(some, top + torch.log(torch.where(some, z, 1.0)), -math.inf)[:, 0]
            cut = lambda x: torch.where(see, x, 0.0).amax(-1, keepdim=True) if length else torch.zeros(n, 1, dtype=torch.float64)  # noqa: E731
            ds = (2 * d + 16) * 2.0 ** -24 * cut(size) + cut(split)
            rel = 4 * ds + 2.0 ** -20 + length * 2.0 ** -22
            spread = p @ vh.abs()
            small = torch.where(see, 2.0 ** -22 * cut(p * s8), 0.0) @ torch.where(seen, cv[:, h // g], 0.0).abs() if length else 0.0
            out[lo:hi, h], lse[lo:hi, h] = o, log
            eo[lo:hi, h] = u * o.abs() + (1 + u) * ((u + rel) * spread + small) + ref.smallest(dt)
            el[lo:hi, h] = (2 * ds[:, 0] + 2.0 ** -20 + length * 2.0 ** -22 + 2.0 ** -22 * torch.where(some[:, 0], log.abs(), 0.0))
    return out, lse, eo, el
