"""ar_qk_norm_rope against the formula in 64 bits: head sizes, strides, pairings, axes, cache slots."""
import math
from fractions import Fraction

import pytest
import torch

import serve_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    import tensor_all_reduce_gb300 as tar
    with tar.Context(0) as c:
        yield c


def freqs(half, base=10000.0):
    return (base ** (-torch.arange(half, dtype=torch.float64) / max(half, 1))).float()


def cut(half, axes):
    return [half // axes + (1 if i < half % axes else 0) for i in range(axes)]


def make(tokens, hq, hk, d, dtype, rot, axes=1, far=5000, norm=True, page=16, seed=0):
    g = torch.Generator().manual_seed(seed)
    t = ref.DT[dtype]
    rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    qkv = (rand(tokens, hq + 2 * hk, d) * 2).to(t)
    blocks = -(-tokens // page) + 2
    slots = torch.randperm(blocks * page, generator=g)[:tokens]
    return dict(qkv=qkv, q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:], freq=freqs(rot // 2),
                pos=torch.randint(0, far, (axes, tokens), generator=g, dtype=torch.int32),
                wq=(rand(d) * 0.2 + 1.0).to(t) if norm else None, wk=(rand(d) * 0.2 + 1.0).to(t) if norm else None, slots=slots,
                kc=rand(blocks, page, hk, d).to(t), vc=rand(blocks, page, hk, d).to(t))


def on_gpu(x):
    """The tensors on the GPU; q, k and v are views of the packed projection there too."""
    b, hq, hk = x["qkv"].cuda(), x["q"].shape[1], x["k"].shape[1]
    out = {n: t.cuda() if t is not None else None for n, t in x.items()}
    out.update(qkv=b, q=b[:, :hq], k=b[:, hq:hq + hk], v=b[:, hq + hk:])
    return out


def near(got, want, bound):
    err = (got.cpu().double() - want).abs()
    assert (err <= bound).all(), f"{(err - bound).max().item():.3g} over, at {torch.argmax(err - bound).item()}, of {want.abs().max().item():.3g}"


def check(ctx, x, gemma=False, pairs=False, sections=None, dealt=False, eps=1e-6):
    axis = ref.axis_of(sections, dealt) if sections else [0] * x["freq"].numel()
    wq, eq = ref.rope(x["q"], x["wq"], eps, gemma, x["pos"], x["freq"], pairs, axis)
    wk, ek = ref.rope(x["k"], x["wk"], eps, gemma, x["pos"], x["freq"], pairs, axis)
    y = on_gpu(x)
    freq = y["freq"] if y["freq"].numel() else None
    qo, ko = ctx.qk_norm_rope(y["q"], y["k"], y["v"], y["pos"] if sections else y["pos"][0], freq, q_weight=y["wq"], k_weight=y["wk"], eps=eps,
                              gemma=gemma, pairs=pairs, sections=sections, dealt=dealt, k_cache=y["kc"], v_cache=y["vc"], slots=y["slots"])
    torch.cuda.synchronize()
    assert ctx.device_status() == 0
    near(qo, wq, eq)
    near(ko, wk, ek)
    there = x["slots"] >= 0
    at = x["slots"][there]
    kc, vc = y["kc"].cpu().flatten(0, 1), y["vc"].cpu().flatten(0, 1)
    assert torch.equal(kc[at], ko.cpu()[there])
    assert torch.equal(vc[at], x["v"][there])
    rest = torch.ones(kc.shape[0], dtype=torch.bool)
    rest[at] = False
    assert torch.equal(kc[rest], x["kc"].flatten(0, 1)[rest]) and torch.equal(vc[rest], x["vc"].flatten(0, 1)[rest])
    return qo, ko


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("d, rot", [(64, 64), (80, 80), (96, 48), (128, 128), (128, 32), (256, 256), (256, 64), (8, 8), (72, 40), (128, 20), (48, 0),
                                    (2, 2), (33, 32), (1, 0), (250, 250)])
def test_head_sizes(ctx, dtype, pairs, d, rot):
    check(ctx, make(37, 6, 2, d, dtype, rot, seed=d + rot), pairs=pairs, gemma=pairs)


@pytest.mark.parametrize("tokens", [1, 2, 5, 16, 333, 2049])
@pytest.mark.parametrize("hq, hk", [(12, 2), (1, 1), (7, 1), (48, 8), (3, 5)])
def test_tokens_and_heads(ctx, tokens, hq, hk):
    check(ctx, make(tokens, hq, hk, 128, "bf16", 128, seed=tokens))


@pytest.mark.parametrize("tokens", [460, 1001, 1501, 2203, 2705, 3101, 3501])
@pytest.mark.parametrize("hq, hk, d, rot, pairs", [(4, 2, 64, 64, False), (4, 2, 80, 80, True), (2, 1, 96, 24, False), (3, 1, 256, 72, False)])
def test_units_of_several_tokens(ctx, tokens, hq, hk, d, rot, pairs):
    """Short rows: two to eight tokens are staged together, the last unit is not full, some have no slot."""
    x = make(tokens, hq, hk, d, "bf16", rot, axes=2, seed=tokens)
    x["slots"][::7] = -1
    check(ctx, x, sections=[rot // 2 - 3, 3], dealt=pairs, pairs=pairs)


@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("dealt", [False, True])
@pytest.mark.parametrize("d, pairs", [(128, False), (80, True)])
def test_axes(ctx, axes, dealt, d, pairs):
    x = make(50, 4, 2, d, "bf16", d, axes=axes, seed=axes)
    check(ctx, x, sections=cut(d // 2, axes), dealt=dealt, pairs=pairs)


def test_uneven_and_empty_sections(ctx):
    for sections in ([16, 24, 24], [0, 64, 0], [64, 0, 0], [1, 1, 62]):
        for dealt in (False, True):
            check(ctx, make(20, 4, 2, 128, "fp16", 128, axes=3, seed=3), sections=sections, dealt=dealt)


def test_far_positions(ctx):
    x = make(64, 4, 2, 128, "bf16", 128, far=1 << 20, seed=9)
    x["pos"][0, 0], x["pos"][0, 1] = (1 << 20) + 1, -(1 << 20)
    check(ctx, x)


def test_farthest_positions(ctx):
    """At 2^31 a binary64 product of position and frequency is off by 2^-22 of a radian, more than the
    kernel's angle: the expected angles come from exact fractions, with pi by Machin's formula."""
    x = make(64, 4, 2, 128, "bf16", 128, far=(1 << 31) - 1, seed=9)
    x["pos"][0, 0], x["pos"][0, 1] = (1 << 31) - 1, -(1 << 31)

    def arctan_inv(n):
        return sum(Fraction((-1) ** k, (2 * k + 1) * n ** (2 * k + 1)) for k in range(90))
    two_pi = Fraction(round(2 * (16 * arctan_inv(5) - 4 * arctan_inv(239)) * 2 ** 220), 2 ** 220)
    turns = [[float((Fraction(p) * Fraction(f) / two_pi) % 1) for f in x["freq"].tolist()] for p in x["pos"][0].tolist()]
    theta = (torch.tensor(turns, dtype=torch.float64) * 2 * math.pi)[:, None]
    g = on_gpu(x)
    got = ctx.qk_norm_rope(g["q"], g["k"], None, g["pos"][0], g["freq"], q_weight=g["wq"], k_weight=g["wk"])
    for y, n, w in zip(got, ("q", "k"), ("wq", "wk")):
        z, _ = ref.rope(x[n], x[w], 1e-6, False, None, None, False, [])
        a, b = z[..., :64], z[..., 64:]
        want = torch.cat([a * theta.cos() - b * theta.sin(), b * theta.cos() + a * theta.sin()], -1)
        size = (a.abs() + b.abs()).repeat(1, 1, 2) * 2.0 ** -19
        near(y, want, ref.half_step(x[n].dtype) * (want.abs() + size) + size + ref.smallest(x[n].dtype))


def test_without_norm_or_rotation(ctx):
    check(ctx, make(33, 4, 2, 128, "bf16", 128, norm=False))
    check(ctx, make(33, 4, 2, 128, "bf16", 0, norm=True))
    x = make(33, 4, 2, 128, "bf16", 0, norm=False)
    qo, _ = check(ctx, x)
    assert torch.equal(qo.cpu(), x["q"])
    x = make(33, 4, 2, 64, "bf16", 64)
    x["wq"] = None  # one of the two
    check(ctx, x)


def test_padding_slots(ctx):
    x = make(40, 4, 2, 128, "bf16", 128)
    x["slots"][3] = -1
    x["slots"][-5:] = -1
    check(ctx, x)


def test_slots_out_of_range_are_dropped(ctx):
    x = on_gpu(make(40, 4, 2, 128, "bf16", 128))
    before = x["kc"].clone(), x["vc"].clone()
    slots = torch.full_like(x["slots"], -1)
    slots[0], slots[1], slots[2] = x["kc"].shape[0] * 16, -2, 1 << 40
    ctx.qk_norm_rope(x["q"], x["k"], x["v"], x["pos"][0], x["freq"], k_cache=x["kc"], v_cache=x["vc"], slots=slots)
    assert ctx.device_status() == 2 and ctx.device_status() == 0
    assert torch.equal(before[0], x["kc"]) and torch.equal(before[1], x["vc"])


def test_in_place_on_a_packed_projection(ctx):
    x = make(70, 12, 2, 128, "bf16", 128)
    g = on_gpu(x)
    ctx.qk_norm_rope(g["q"], g["k"], g["v"], g["pos"][0], g["freq"], q_weight=g["wq"], k_weight=g["wk"], q_out=g["q"], k_out=g["k"])
    h = on_gpu(x)
    q2, k2 = ctx.qk_norm_rope(h["q"], h["k"], None, h["pos"][0], h["freq"], q_weight=h["wq"], k_weight=h["wk"])
    assert torch.equal(g["q"], q2) and torch.equal(g["k"], k2) and torch.equal(g["v"].cpu(), x["v"])


def test_only_q_and_only_k(ctx):
    g = on_gpu(make(30, 4, 4, 96, "fp16", 96))
    qo, ko = ctx.qk_norm_rope(g["q"], g["k"], None, g["pos"][0], g["freq"], q_weight=g["wq"], k_weight=g["wk"])
    q1, none = ctx.qk_norm_rope(g["q"], None, None, g["pos"][0], g["freq"], q_weight=g["wq"])
    assert none is None and torch.equal(q1, qo)
    none, k1 = ctx.qk_norm_rope(None, g["k"], None, g["pos"][0], g["freq"], k_weight=g["wk"])
    assert none is None and torch.equal(k1, ko)


@pytest.mark.parametrize("shift", [1, 4])
def test_unaligned_rows(ctx, shift):
    """Rows that start off a 16-byte boundary, with odd strides."""
    x = make(21, 5, 3, 64, "bf16", 64)
    g = on_gpu(x)

    def odd(t):
        n, h, d = t.shape
        buf = torch.zeros(n * (h * (d + 3) + 5) + 8, dtype=t.dtype, device="cuda")
        v = buf[shift:shift + n * (h * (d + 3) + 5)].view(n, -1)[:, :h * (d + 3)].unflatten(1, (h, d + 3))[..., :d]
        v.copy_(t)
        return v
    got = ctx.qk_norm_rope(odd(g["q"]), odd(g["k"]), None, g["pos"][0], g["freq"], q_weight=g["wq"], k_weight=g["wk"],
                           q_out=odd(g["q"]), k_out=odd(g["k"]))
    for y, n, w in zip(got, ("q", "k"), ("wq", "wk")):
        near(y, *ref.rope(x[n], x[w], 1e-6, False, x["pos"], x["freq"], False, [0] * 32))


def test_cache_orders(ctx):
    """Heads before tokens in the block, and k and v in one tensor."""
    g = on_gpu(make(40, 4, 2, 128, "bf16", 128))
    ko = ctx.qk_norm_rope(g["q"], g["k"], g["v"], g["pos"][0], g["freq"], k_cache=g["kc"], v_cache=g["vc"], slots=g["slots"])[1]
    one = torch.zeros(g["kc"].shape[0], 2, 2, 16, 128, dtype=torch.bfloat16, device="cuda")  # block, k or v, head, token, dim
    kc, vc = one[:, 0].transpose(1, 2), one[:, 1].transpose(1, 2)
    ctx.qk_norm_rope(g["q"], g["k"], g["v"], g["pos"][0], g["freq"], k_cache=kc, v_cache=vc, slots=g["slots"])
    at = g["slots"]
    assert torch.equal(kc[at // 16, at % 16], ko) and torch.equal(vc[at // 16, at % 16], g["v"])


def test_tiny_and_huge_values(ctx):
    x = make(16, 2, 2, 128, "bf16", 128)
    x["q"][0], x["q"][1], x["q"][2] = 0.0, 1e-20, 1e15
    check(ctx, x)


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("d, rot", [(128, 64), (80, 40), (33, 32)])
def test_an_infinity_stays_in_its_pair(ctx, pairs, d, rot):
    """Without a norm an infinity reaches its own pair only; an element that does not turn keeps it."""
    x = make(9, 2, 1, d, "bf16", rot, norm=False)
    x["q"][3, 1, rot:] = float("inf")
    x["q"][4, 0, 5] = float("inf")
    g = on_gpu(x)
    qo = ctx.qk_norm_rope(g["q"], None, None, g["pos"][0], g["freq"], pairs=pairs)[0].cpu()
    other = 4 if pairs else 5 + rot // 2
    bad = ~torch.isfinite(qo)
    want = torch.zeros_like(bad)
    want[3, 1, rot:] = True
    want[4, 0, 5] = want[4, 0, other] = True
    assert torch.equal(bad, want) and (qo[3, 1, rot:] == float("inf")).all()


@pytest.mark.parametrize("hq, hk, d", [(48, 8, 128), (5, 3, 64), (9, 2, 256), (16, 16, 80)])
def test_both_forms_agree(ctx, hq, hk, d):
    """The vector form and the general one, each within the bound, at sizes that share heads and tokens differently."""
    import tensor_all_reduce_gb300 as tar
    for tokens in (1, 3, 160, 1900):
        x = make(tokens, hq, hk, d, "bf16", d, seed=tokens)
        for option, name in ((0, "qk_norm_rope_vec"), (4, "qk_norm_rope_scalar")):
            ctx.set_option(tar.AR_OPT_FORCE_VARIANT, option)
            try:
                check(ctx, x)
                assert ctx.last_variant == name
            finally:
                ctx.set_option(tar.AR_OPT_FORCE_VARIANT, 0)


def test_streams_and_graph(ctx):
    x = on_gpu(make(50, 4, 2, 128, "bf16", 128))
    s = torch.cuda.Stream()
    qo = torch.empty(50, 4, 128, dtype=torch.bfloat16, device="cuda")
    call = lambda: ctx.qk_norm_rope(x["q"], x["k"], x["v"], x["pos"][0], x["freq"], q_weight=x["wq"], k_weight=x["wk"], k_cache=x["kc"],  # noqa: E731
                                    v_cache=x["vc"], slots=x["slots"], q_out=qo, want_k_out=False, stream=s)
    torch.cuda.synchronize()
    call()
    s.synchronize()
    want = qo.clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        call()
    x["pos"].add_(7)
    fresh = ctx.qk_norm_rope(x["q"], None, None, x["pos"][0], x["freq"], q_weight=x["wq"])[0]
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(qo, fresh) and not torch.equal(qo, want)


def test_a_wait_that_runs_out_ends_the_call(ctx):
    """The first copy of each CTA is held back: the call ends with code 1, and the next one is right."""
    import tensor_all_reduce_gb300 as tar
    x = make(3000, 8, 2, 128, "bf16", 128)
    g = on_gpu(x)
    ctx.set_option(tar.AR_OPT_TEST_STALL, 1)
    ctx.set_option(tar.AR_OPT_WAIT_CYCLES, 2000000)
    try:
        ctx.qk_norm_rope(g["q"], g["k"], None, g["pos"][0], g["freq"], q_weight=g["wq"])
        assert ctx.last_variant == "qk_norm_rope_vec" and ctx.device_status() == 1
    finally:
        ctx.set_option(tar.AR_OPT_TEST_STALL, 0)
        ctx.set_option(tar.AR_OPT_WAIT_CYCLES, 0)
    check(ctx, x)


def test_more_heads_than_a_stage_holds(ctx):
    """A token's heads are split over units: 300 q heads of 256, and 100 of 80 with few tokens."""
    check(ctx, make(5, 300, 3, 256, "bf16", 256))
    check(ctx, make(700, 90, 40, 128, "bf16", 64))
    check(ctx, make(2, 100, 7, 80, "fp16", 80), pairs=True)


def test_heads_apart_in_memory(ctx):
    """q of shape [tokens, heads, dim] with a gap between heads, and transposed: each head is fetched by itself."""
    x = make(60, 6, 2, 128, "bf16", 128)
    g = on_gpu(x)
    want = ctx.qk_norm_rope(g["q"], g["k"], None, g["pos"][0], g["freq"], q_weight=g["wq"], k_weight=g["wk"])
    gap = torch.zeros(60, 6, 160, dtype=torch.bfloat16, device="cuda")[..., :128]
    gap.copy_(g["q"])
    turned = g["k"].transpose(0, 1).contiguous().transpose(0, 1)
    got = ctx.qk_norm_rope(gap, g["k"], None, g["pos"][0], g["freq"], q_weight=g["wq"], k_weight=g["wk"])
    assert ctx.last_variant == "qk_norm_rope_vec"
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    import tensor_all_reduce_gb300 as tar
    with pytest.raises(tar.ArError):  # tokens closer than a head: not rows that stand apart
        ctx.qk_norm_rope(None, turned[:, :, :].as_strided((60, 2, 128), (64, 128 * 60, 1)), None, g["pos"][0], g["freq"], k_weight=g["wk"])
    again = ctx.qk_norm_rope(None, turned, None, g["pos"][0], g["freq"], k_weight=g["wk"])[1]
    assert torch.equal(again, want[1])


def test_binding_refuses(ctx):
    x = on_gpu(make(8, 4, 2, 64, "bf16", 64, axes=3))
    with pytest.raises(ValueError):
        ctx.qk_norm_rope(x["q"], x["k"], None, x["pos"], x["freq"])                                  # axes without sections
    with pytest.raises(ValueError):
        ctx.qk_norm_rope(x["q"], x["k"], None, x["pos"][0].long(), x["freq"])
    with pytest.raises(ValueError):
        ctx.qk_norm_rope(x["q"], x["k"].half(), None, x["pos"][0], x["freq"])
    with pytest.raises(ValueError):
        ctx.qk_norm_rope(x["q"].float(), None, None, x["pos"][0], x["freq"])
    with pytest.raises(ValueError):
        ctx.qk_norm_rope(x["q"], x["k"], x["v"], x["pos"][0], x["freq"], k_cache=x["kc"])
    with pytest.raises(ValueError):
        ctx.qk_norm_rope(x["q"], None, None, x["pos"][0], x["freq"], q_weight=x["wq"][:3])
    with pytest.raises(ValueError):
        ctx.qk_norm_rope(None, None, None, x["pos"][0], x["freq"])
