"""ar_paged_append_fp8 against the formula in 64 bits: head sizes, pages, strides, rotations, blocks that hold tokens
already, growing scales, values of any size, both kernel forms."""
import random

import pytest
import torch

import serve8_ref as ref8
import serve_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    import tensor_all_reduce_gb300 as tar
    with tar.Context(0) as c:
        yield c


@pytest.fixture(params=[0, 4], ids=["auto", "general"])
def form(ctx, request):
    import tensor_all_reduce_gb300 as tar
    ctx.set_option(tar.AR_OPT_FORCE_VARIANT, request.param)
    yield request.param
    ctx.set_option(tar.AR_OPT_FORCE_VARIANT, 0)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def cut(half, axes):
    return [half // axes + (1 if i < half % axes else 0) for i in range(axes)]


def make(new, cached, hk, d, dtype="bf16", page=16, rot=None, axes=1, norm=True, seed=0, spare_rows=0, peak=2.0, low=-10, high=-3):
    """Inputs on the CPU: a cache of any codes but NaN's, scales between 2^low and 2^high (powers of two)."""
    g = torch.Generator().manual_seed(seed)
    rng = random.Random(seed)
    t = ref.DT[dtype]
    lens = [c + n for c, n in zip(cached, new)]
    need = [-(-x // page) for x in lens]
    blocks = sum(need) + 3
    ids = list(range(blocks))
    rng.shuffle(ids)
    cols = max(need + [0]) + 1
    table, at = [], 0
    for n in need:
        table.append(ids[at:at + n] + [-1] * (cols - n))
        at += n
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    rows = cu[-1] + spare_rows
    kv = (torch.randn(rows, 2 * hk, d, generator=g) * peak).to(t)
    half = (d // 2 * 2 if rot is None else rot) // 2
    x = dict(kv=kv, hk=hk, table=table, cu=cu, lens=lens, page=page, weight=(torch.randn(d, generator=g) * 0.2 + 1.0).to(t) if norm else None,
             freq=(10000.0 ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float(),
             pos=torch.randint(0, 5000, (axes, rows), generator=g, dtype=torch.int32))
    for n in ("k", "v"):
        c = torch.randint(0, 254, (blocks, page, hk, d), generator=g).to(torch.uint8)
        x[n + "c"] = torch.where(c >= 127, c + 1, c)
        x[n + "s"] = torch.exp2(torch.randint(low, high, (blocks, hk), generator=g).float())
    return x


def states(x):
    return [x[n].cuda() for n in ("kc", "vc", "ks", "vs")]


def call(ctx, x, state, positions, kv=None, **kw):
    kv = x["kv"].cuda() if kv is None else kv
    table = i32(x["table"]) if x["table"] else torch.zeros(0, 1, dtype=torch.int32, device="cuda")
    ctx.paged_append_fp8(kv[:, :x["hk"]], kv[:, x["hk"]:], *state, table, i32(x["cu"]), i32(x["lens"]), positions=positions,
                         inv_freq=x["freq"].cuda() if x["freq"].numel() else None, k_weight=None if x["weight"] is None else x["weight"].cuda(), **kw)
    torch.cuda.synchronize()


def check(ctx, x, gemma=False, pairs=False, sections=None, dealt=False, given=True, kv=None, state=None):
    state = states(x) if state is None else state
    call(ctx, x, state, (x["pos"] if sections else x["pos"][0]).cuda() if given else None, kv, gemma=gemma, pairs=pairs, sections=sections, dealt=dealt)
    assert ctx.device_status() == 0
    verify(x, [t.cpu() for t in state], gemma, pairs, sections, dealt, given)
    return state


def verify(x, after, gemma=False, pairs=False, sections=None, dealt=False, given=True):
    axis = ref.axis_of(sections, dealt) if sections else [0] * x["freq"].numel()
    pos = x["pos"]
    if not given:
        pos = torch.zeros(1, x["kv"].shape[0], dtype=torch.int32)
        for r, length in enumerate(x["lens"]):
            lo, hi = x["cu"][r], x["cu"][r + 1]
            pos[0, lo:hi] = torch.arange(length - (hi - lo), length)
    hk = x["hk"]
    k, ek = ref8.turned(x["kv"][:, :hk], x["weight"], 1e-6, gemma, pos, x["freq"], pairs, axis)
    v = x["kv"][:, hk:].double()
    ref8.check_append([x[n] for n in ("kc", "vc", "ks", "vs")], after, k, v, ek, torch.zeros_like(v), x["table"], x["cu"], x["lens"], x["page"])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("d, rot", [(64, 64), (80, 80), (80, 20), (96, 48), (96, 24), (128, 128), (128, 32), (256, 256), (256, 64), (8, 8), (72, 40),
                                    (128, 20), (48, 0), (2, 2), (33, 32), (1, 0), (250, 250), (16, 6)])
def test_head_sizes(ctx, form, dtype, pairs, d, rot):
    check(ctx, make([1, 37, 0, 5], [40, 3, 9, 0], 3, d, dtype, rot=rot, seed=d + rot), pairs=pairs, gemma=pairs)


@pytest.mark.parametrize("page", [1, 2, 5, 8, 16, 24, 32, 64, 100, 128, 256, 300, 1000])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_page_sizes(ctx, form, page, d):
    check(ctx, make([1, 140, 1, 300, 7], [700, 5, 64, page - 1, page], 2, d, page=page, seed=page))
    check(ctx, make([1, 2 * page + 1], [3, 2], 1, d, "fp16", page=page, seed=page, norm=False), pairs=True)


@pytest.mark.parametrize("hk", [1, 2, 3, 5, 8, 16, 40])
@pytest.mark.parametrize("new", [[1], [1] * 9, [17, 1, 1, 33], [400]])
def test_heads(ctx, form, hk, new):
    check(ctx, make(new, [11 * i % 50 for i in range(len(new))], hk, 64, seed=hk))


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("dealt", [False, True])
@pytest.mark.parametrize("d, pairs", [(128, False), (80, True)])
def test_axes(ctx, form, axes, dealt, d, pairs):
    x = make([30, 1, 19], [5, 16, 0], 2, d, axes=axes, seed=axes)
    check(ctx, x, sections=cut(d // 2, axes), dealt=dealt, pairs=pairs)
    row = x["pos"][:1]
    x["pos"] = row.expand(axes, -1)  # one row that all axes share
    check(ctx, x, sections=cut(d // 2, axes), dealt=dealt, pairs=pairs)


def test_places_are_the_default_positions(ctx, form):
    check(ctx, make([30, 1, 19, 0], [5, 160, 0, 7], 2, 128, seed=3), given=False)
    check(ctx, make([1, 1], [100000, 20], 1, 64, seed=4), given=False)


@pytest.mark.parametrize("norm, rot", [(False, 0), (True, 0), (False, None)])
def test_without_norm_or_rotation(ctx, form, norm, rot):
    check(ctx, make([30, 1, 19], [5, 160, 0], 2, 128, norm=norm, rot=rot, seed=3))


def test_scales_that_grow_and_stay(ctx, form):
    """Held codes are rounded to a scale that grew, keep their bits under one that did not."""
    for low, high in ((-30, -20), (-8, -4), (3, 8), (-32, -30)):
        x = make([1, 1, 3, 20], [1, 15, 40, 7], 4, 128, seed=low, low=low, high=high)
        check(ctx, x)
    x = make([1, 1, 1], [1, 15, 40], 2, 64, seed=5)
    x["ks"] *= 1.3  # a scale of another kind: kept where it is large enough, else grown to a power of two
    x["ks"][:, 0] *= 2.0 ** 10
    state = states(x)
    call(ctx, x, state, x["pos"][0].cuda())
    for r, length in enumerate(x["lens"]):
        b = x["table"][r][(length - 1) // 16]
        assert state[2][b, 0].item() == x["ks"][b, 0].item()
        held = (length - 1) % 16
        assert torch.equal(state[0][b, :held, 0].cpu(), x["kc"][b, :held, 0])


def test_scales_outside_their_range(ctx, form):
    x = make([1] * 6, [5] * 6, 1, 64, seed=5)
    odd = [0.0, -1.0, float("nan"), float("inf"), 2.0 ** 100, 1e-42]
    for r, s in enumerate(odd):
        b = x["table"][r][0]
        x["vs"][b] = x["ks"][b] = s
    state = states(x)
    call(ctx, x, state, x["pos"][0].cuda())
    assert ctx.device_status() == 0
    for r, s in enumerate(odd):
        b = x["table"][r][0]
        if s > 1:
            assert state[3][b].item() == state[2][b].item() == 2.0 ** 32
        else:
            top = x["kv"][r, 1].double().abs().max().item()
            assert state[3][b].item() == ref8.fresh(top)
            assert torch.equal(state[1][b, 5, 0].cpu().view(ref8.E4M3).double(), ref8.round_e4m3(x["kv"][r, 1].double() / ref8.fresh(top)))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_values_of_any_size(ctx, form, dtype):
    """Borders of a scale, ties of the codes, subnormal and largest values, zeros, infinities and NaN."""
    x = make([9, 1, 1, 1, 1, 1], [3, 0, 1, 2, 3, 20], 2, 64, dtype, rot=0, norm=False, seed=6)
    t = x["kv"].dtype
    kv = x["kv"]
    kv[9] = 0.0
    kv[10, :, 3:] = 0.0
    kv[10, 0, :3] = torch.tensor([448.0, 14.0, 0.4375]).to(t)       # 448 2^k exactly
    kv[10, 1, :3] = torch.tensor([448.0, 2.0 ** -10, 3 * 2.0 ** -10]).to(t)  # ties of the smallest codes
    kv[11, 0, 0], kv[11, 1, 5] = float("inf"), float("nan")
    kv[12] = torch.finfo(t).max
    kv[13] = torch.finfo(t).tiny * torch.finfo(t).eps
    kv[13, 2, 7] = float("-inf")
    kv[0, 0, 0], kv[0, 1, 0] = 450.0, 449.0
    check(ctx, x)
    y = dict(x, weight=torch.ones(64, dtype=t))
    y["kv"] = kv.clone()
    y["kv"][11:14] = 1.0
    check(ctx, y)


def test_the_same_tokens_twice(ctx, form):
    """A step run again gives the same cache."""
    x = make([20, 1, 1], [5, 160, 7], 2, 128, seed=3)
    state = check(ctx, x)
    again = [t.clone() for t in state]
    call(ctx, x, again, x["pos"][0].cuda())
    assert all(torch.equal(a, b) for a, b in zip(state, again))


def test_token_by_token(ctx, form):
    """Tokens added one at a time and at once: equal where no scale grew twice over a held token, near everywhere."""
    n, page = 40, 16
    x = make([n], [0], 2, 64, page=page, seed=8)
    once = check(ctx, x)
    state = states(x)
    for i in range(n):
        y = dict(x, kv=x["kv"][i:i + 1], pos=x["pos"][:, i:i + 1], cu=[0, 1], lens=[i + 1])
        call(ctx, y, state, y["pos"][0].cuda())
    used = x["table"][0][:3]
    for which in (0, 1):
        assert torch.equal(state[which + 2][used], once[which + 2][used])
        a, b = (ref8.values(s[which][used].cpu(), s[which + 2][used].cpu()).flatten(0, 1)[:n] for s in (state, once))
        # a code of the last scale, and one rounded through finer ones: powers of two, so apart only below 2^-6 of a
        # scale, where each of at most 20 roundings moves it by half a step of 2^-9
        s = once[which + 2][used].cpu().double().repeat_interleave(page, 0)[:n, :, None]
        assert ((a - b).abs() <= 20 * 2.0 ** -10 * s).all()


def test_empty_calls(ctx, form):
    x = make([0, 0], [5, 0], 2, 64, spare_rows=3)
    state = check(ctx, x)
    assert all(torch.equal(s.cpu(), x[n]) for s, n in zip(state, ("kc", "vc", "ks", "vs")))
    check(ctx, make([], [], 2, 64, spare_rows=3))
    assert ctx.last_variant == "none"
    check(ctx, make([0, 0, 2, 0], [0, 9, 2, 0], 4, 64, spare_rows=5))


def test_many_requests(ctx, form):
    check(ctx, make([1] * 700, [i % 37 for i in range(700)], 1, 64, page=8, seed=8))
    new = [(1, 0, 2, 0, 0, 30)[i % 6] for i in range(2000)]  # several rounds of requests a CTA's threads
    check(ctx, make(new, [i % 41 for i in range(2000)], 1, 64, page=8, seed=9))


def test_rows_that_begin_behind_the_first(ctx, form):
    x = make([3, 0, 50], [40, 5, 30], 2, 64, seed=18)
    x["kv"] = torch.cat([x["kv"][:7], x["kv"]])
    x["pos"] = torch.cat([x["pos"][:, :7], x["pos"]], 1)
    x["cu"] = [c + 7 for c in x["cu"]]
    check(ctx, x)


def test_what_is_out_of_range_is_dropped(ctx, form):
    """Block numbers outside the cache, tokens behind the table, lengths below the new tokens, rows behind the end:
    dropped with code 2, the others are written."""
    base = make([20, 3, 5, 2], [12, 30, 0, 7], 2, 64, seed=12)
    blocks = base["kc"].shape[0]

    def go(x, drop):
        """`drop`: (request, tokens that are written) of the requests that lose some."""
        state = states(x)
        call(ctx, x, state, x["pos"][0].cuda())
        assert ctx.device_status() == 2
        return [t.cpu() for t in state]

    for bad in (-1, -5, blocks, 1 << 30, 2 ** 31 - 1, -2 ** 31):
        x = dict(base, table=[list(t) for t in base["table"]])
        x["table"][0][1] = bad  # tokens 16 .. 31 of request 0
        after = go(x, None)
        y = dict(base, cu=[0, 4, 20, 23, 28, 30], lens=[16, 0, 33, 5, 9])  # request 0 up to place 16; rows 4 .. 19 nobody's
        y["table"] = [base["table"][0], [], *base["table"][1:]]
        y["cu"], y["lens"], y["table"] = [0, 4, 4, 7, 12, 14], [16, 0, 33, 5, 9], y["table"]
        keep = list(range(4)) + list(range(20, 30))
        y["kv"], y["pos"] = base["kv"][keep], base["pos"][:, keep]
        y["table"][1] = [-1] * len(base["table"][0])
        verify(y, after)
    # a table of two columns holds 32 tokens: request 1 (places 30 .. 32) loses its last
    x = dict(base, table=[t[:2] for t in base["table"]])
    after = go(x, None)
    keep = [i for i in range(30) if i != 22]
    verify(dict(base, kv=base["kv"][keep], pos=base["pos"][:, keep], cu=[0, 20, 22, 27, 29], lens=[32, 32, 5, 9]), after)
    # lengths below the new tokens: the request is dropped
    for length in (2, -1, -2 ** 31):
        x = dict(base, lens=[32, length, 5, 9])
        after = go(x, None)
        keep = [i for i in range(30) if not 20 <= i < 23]
        verify(dict(base, kv=base["kv"][keep], pos=base["pos"][:, keep], cu=[0, 20, 20, 25, 27], lens=[32, 0, 5, 9]), after)
    # row ranges behind the rows are cut: request 3 has fewer tokens, which end at its length
    x = dict(base, cu=[0, 20, 23, 28, 90])
    after = go(x, None)
    verify(base, after)


def test_orders_and_strides(ctx, form):
    """k and v apart and between each other, caches and scales in other orders, off 16-byte boundaries: the same codes."""
    x = make([20, 1, 70], [300, 129, 0], 4, 64, seed=14)
    want = [t.cpu() for t in check(ctx, x)]
    blocks, page, hk, d = x["kc"].shape
    a = x["pos"][0].cuda()
    freq, w = x["freq"].cuda(), x["weight"].cuda()
    args = (i32(x["table"]), i32(x["cu"]), i32(x["lens"]))
    kv = x["kv"].cuda()
    wide = torch.zeros(kv.shape[0], hk, 2, d, dtype=kv.dtype, device="cuda")
    wide[:, :, 0], wide[:, :, 1] = kv[:, :hk], kv[:, hk:]
    odd = torch.zeros(kv.numel() + 1, dtype=kv.dtype, device="cuda")[1:].view(kv.shape)
    odd.copy_(kv)
    for k, v in ((wide[:, :, 0], wide[:, :, 1]), (odd[:, :hk], odd[:, hk:])):
        for order in ("btwh", "bthw", "bhtw", "wbht", "whbt"):  # block, token, head, which
            size = dict(b=blocks, t=page, h=hk, w=2)
            one = torch.zeros([size[n] for n in order] + [d], dtype=torch.uint8, device="cuda")
            turned = one.permute(*[order.index(n) for n in "wbth"], 4)
            turned[0].copy_(x["kc"].cuda())
            turned[1].copy_(x["vc"].cuda())
            sc = torch.stack([x["ks"], x["vs"]]).cuda().permute(2, 1, 0).contiguous()  # [head, block, which]
            ctx.paged_append_fp8(k, v, turned[0].view(torch.float8_e4m3fn), turned[1].view(torch.float8_e4m3fn), sc[..., 0].t(), sc[..., 1].t(), *args,
                                 positions=a, inv_freq=freq, k_weight=w)
            assert torch.equal(turned[0].cpu(), want[0]) and torch.equal(turned[1].cpu(), want[1])
            assert torch.equal(sc[..., 0].t().cpu(), want[2]) and torch.equal(sc[..., 1].t().cpu(), want[3])
    # caches off a boundary, rows with padding
    for off, pad in ((1, 0), (4, 4), (8, 8), (0, 5)):
        bufs = [torch.zeros(off + blocks * page * hk * (d + pad), dtype=torch.uint8, device="cuda") for _ in range(2)]
        caches = [b[off:].view(blocks, page, hk, d + pad)[..., :d] for b in bufs]
        for c, n in zip(caches, ("kc", "vc")):
            c.copy_(x[n].cuda())
        ks, vs = x["ks"].cuda(), x["vs"].cuda()
        ctx.paged_append_fp8(kv[:, :hk], kv[:, hk:], *caches, ks, vs, *args, positions=a, inv_freq=freq, k_weight=w)
        got = [t.cpu() for t in (*caches, ks, vs)]
        assert all(torch.equal(g, z) for g, z in zip(got, want))
    assert ctx.device_status() == 0


def test_captured_call_follows_the_lengths(ctx, form):
    x = make([1, 1, 2], [700, 15, 31], 2, 128, seed=15)
    state = states(x)
    kv, pos, table, cu, lens = x["kv"].cuda(), x["pos"][0].cuda(), i32(x["table"]), i32(x["cu"]), i32(x["lens"])
    freq, w = x["freq"].cuda(), x["weight"].cuda()
    args = (kv[:, :2], kv[:, 2:], *state, table, cu, lens)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        ctx.paged_append_fp8(*args, positions=pos, inv_freq=freq, k_weight=w)
    for new, total in (([1, 1, 2], [701, 16, 33]), ([4, 0, 0], [13, 16, 3]), ([0, 1, 1], [700, 1, 17])):
        for t, n in zip(state, ("kc", "vc", "ks", "vs")):
            t.copy_(x[n])
        edges = [0]
        for n in new:
            edges.append(edges[-1] + n)
        cu.copy_(i32(edges))
        lens.copy_(i32(total))
        g.replay()
        torch.cuda.synchronize()
        assert ctx.device_status() == 0
        verify(dict(x, cu=edges, lens=total), [t.cpu() for t in state])


def test_offsets_beyond_32_bits(ctx, form):
    page, hk, d = 64, 8, 128
    blocks = (1 << 32) // (page * hk * d) + 200
    small = make([70], [60], hk, d, page=page, seed=16)
    state = [torch.zeros(blocks, page, hk, d, dtype=torch.uint8, device="cuda") for _ in range(2)] + [torch.ones(blocks, hk, device="cuda") for _ in range(2)]
    near, far = small["table"][0][:3], [blocks - 1 - b for b in small["table"][0][:3]]
    for t, n in zip(state, ("kc", "vc", "ks", "vs")):
        t[far] = small[n][near].cuda()
    call(ctx, dict(small, table=[far]), state, small["pos"][0].cuda())
    after = [small[n].clone() for n in ("kc", "vc", "ks", "vs")]
    for a, t in zip(after, state):
        a[near] = t[far].cpu()
    verify(small, after)


def test_binding_refuses(ctx):
    import tensor_all_reduce_gb300 as tar
    x = make([2], [20], 2, 64)
    kv, (kc, vc, ks, vs) = x["kv"].cuda(), states(x)
    k, v, t, cu, lens, pos, freq = kv[:, :2], kv[:, 2:], i32(x["table"]), i32(x["cu"]), i32(x["lens"]), x["pos"].cuda(), x["freq"].cuda()
    f = ctx.paged_append_fp8
    before = [s.clone() for s in (kc, vc, ks, vs)]
    for bad in (lambda: f(k.float(), v, kc, vc, ks, vs, t, cu, lens), lambda: f(k, v[:, :1], kc, vc, ks, vs, t, cu, lens),
                lambda: f(k, v.half(), kc, vc, ks, vs, t, cu, lens), lambda: f(k, v, kc.half(), vc, ks, vs, t, cu, lens),
                lambda: f(k, v, kc, vc[1:], ks, vs, t, cu, lens), lambda: f(k, v, kc, vc, ks[1:], vs, t, cu, lens),
                lambda: f(k, v, kc, vc, ks, vs.double(), t, cu, lens), lambda: f(k, v, kc, vc, ks, vs, t, cu[:1], lens),
                lambda: f(k, v, kc, vc, ks, vs, t, cu, lens, positions=pos[0, :1], inv_freq=freq),
                lambda: f(k, v, kc, vc, ks, vs, t, cu, lens, inv_freq=freq, sections=[16, 16]),
                lambda: f(k, v, kc, vc, ks, vs, t, cu, lens, k_weight=ks)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: f(k, v, kc, kc, ks, vs, t, cu, lens), lambda: f(k, v, kc, vc, ks, ks, t, cu, lens),
                lambda: f(k, v, kc, vc, ks, vs[:1].expand(vs.shape), t, cu, lens), lambda: f(k, v, kc, vc, ks, vs, t, cu, lens, eps=-1.0)):
        with pytest.raises(tar.ArError):
            bad()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, (kc, vc, ks, vs)))


def test_forms(ctx):
    """Which form serves which call."""
    import tensor_all_reduce_gb300 as tar
    for d, rot, pairs, want in ((128, 128, False, "vec"), (80, 80, True, "vec"), (80, 20, False, "scalar"), (80, 20, True, "vec"), (64, 0, False, "vec"),
                                (256, 64, False, "vec"), (8, 8, False, "vec"), (36, 8, False, "scalar")):
        check(ctx, make([3, 20], [5, 0], 2, d, rot=rot), pairs=pairs)
        assert ctx.last_variant == "paged_append_fp8_" + want
    ctx.set_option(tar.AR_OPT_FORCE_VARIANT, 4)
    check(ctx, make([3], [50], 2, 128))
    assert ctx.last_variant == "paged_append_fp8_scalar"
    ctx.set_option(tar.AR_OPT_FORCE_VARIANT, 0)
