"""ar_paged_attention_fp8 where a product of 0 or a small weight is easily lost: NaN codes in blocks that no row sees, rows of huge
queries, one weight far above very many others, errors over long contexts."""
import math

import pytest
import torch

import serve8_ref as ref8
import serve_ref as ref
import test_gpu_paged_attention_fp8 as pa8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    import tensor_all_reduce_gb300 as tar
    with tar.Context(0) as c:
        yield c


@pytest.fixture(params=["auto", "general"])
def form(ctx, request):
    import tensor_all_reduce_gb300 as tar
    ctx.set_option(tar.AR_OPT_FORCE_VARIANT, 4 if request.param == "general" else 0)
    yield request.param
    ctx.set_option(tar.AR_OPT_FORCE_VARIANT, 0)


# new tokens of four requests, and the form that serves them with two q heads a key head
FEW = [1, 4, 6, 1], "few"
LARGER = [1, 7, 20, 3], "few"
DRAFTS = [1, 30, 60, 9], "tma"
CHUNKS = [1, 4, 300, 200], "tma"
BATCHES = [FEW, LARGER, DRAFTS, CHUNKS]


def served_by(ctx, form, name):
    assert ctx.last_variant == "paged_attention_fp8_" + ("mma" if form == "general" else name)


@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("prefix", [0, 70])
@pytest.mark.parametrize("page, d, dtype", [(8, 64, "bf16"), (16, 128, "fp16"), (24, 128, "bf16"), (16, 256, "bf16"), (64, 256, "fp16"), (1, 64, "bf16")])
def test_released_blocks_may_hold_nan(ctx, form, batch, prefix, page, d, dtype):
    """A block that no row sees may be another request's by now, or unwritten: NaN codes of keys and values and any scale in it stay
    its own, inside a tile that rows see the rest of too."""
    (new, name), window, lens = batch, 100, [1900, 700, 1300, 290]
    x = pa8.make(new, lens, 4, 2, d, dtype, page=page, seed=page)  # what no request holds is NaN
    kw = dict(window=window)
    if prefix:
        kw["prefix_lens"] = torch.full((4,), prefix, dtype=torch.int32)
    spare = next(b for b in range(x["kc"].shape[0]) if not any(b in t for t in x["table"]))
    x["ks"][spare], x["vs"][spare] = float("inf"), float("nan")
    for row, n, length in zip(x["table"], new, lens):
        low = max(length - n - window + 1, 0)
        for j in range(-(-prefix // page), low // page):
            row[j] = spare
    pa8.check(ctx, x, **kw)
    if page > 1:
        served_by(ctx, form, name)
    pa8.check(ctx, x, causal=False, **kw)


@pytest.mark.parametrize("batch", BATCHES)
@pytest.mark.parametrize("d", [128, 256])
def test_products_of_zero_with_huge_queries(ctx, form, batch, d):
    """A key of zeros scores 0 against a row of any size under a scale of its own of any size, whatever bends the scores: its weight is
    that of a score of 0, beside keys whose scores the cap bounds.  Scores are 0 and the cap, in 32 bits up to 2^-18 of log2
    units (a cap of 5: 2^-22 of it, tanh from an exponential and a reciprocal), so weights to 2^-18 relative, then rounded."""
    new, name = batch
    lens = [n + 90 for n in new]
    x = pa8.make(new, lens, 4, 2, d, "bf16", seed=3, garbage=0, even=True)
    x["q"] = torch.where(torch.rand(x["q"].shape, generator=torch.Generator().manual_seed(1)) < 0.5, 2.0 ** 120, 2.0 ** 119).to(x["q"].dtype)
    x["ks"].fill_(2.0 ** 16)
    zero = x["kc"].clone().zero_()
    slopes = torch.tensor([0.5, 0.25, 0.0, 1.5])
    for kw in (dict(slopes=slopes), dict(softcap=5.0), dict(softcap=100.0), dict(softcap=5.0, slopes=slopes), dict(scale=-0.3), dict(scale=0.0)):
        pa8.check(ctx, dict(x, kc=zero), **kw)
        served_by(ctx, form, name)
    # every third key points along the queries: scores of 0 and of the cap
    x["kc"] = zero.clone()
    flat = torch.zeros(x["kc"].shape[0], x["kc"].shape[1], dtype=torch.bool)
    for row, length in zip(x["table"], lens):
        for j in range(0, length, 3):
            flat[row[j // 16], j % 16] = True
    x["kc"][flat] = pa8.code(2.0)
    out, _ = pa8.run(ctx, x, scale=d ** -0.5, softcap=5.0)
    u = ref.half_step(torch.bfloat16)
    for r, length in enumerate(lens):
        j = torch.arange(length)
        at = torch.tensor(x["table"][r])[j // 16], j % 16
        v = x["vc"][at].view(ref8.E4M3).double() * x["vs"].double()[at[0]][..., None]  # [length, 2, d]
        pos = torch.arange(length - new[r], length)[:, None]
        w = torch.where(j <= pos, torch.where(j % 3 == 0, math.exp(5.0), 1.0).double(), 0.0)
        p = w / w.sum(-1, keepdim=True)
        for h in range(4):
            o, spread = p @ v[:, h // 2], p @ v[:, h // 2].abs()
            got = out[x["cu"][r]:x["cu"][r + 1], h].double()
            assert ((got - o).abs() <= u * o.abs() + (1 + u) * (u + 2.0 ** -16) * spread + ref.smallest(torch.bfloat16)).all()


# the relative error of a weight, by form
def weight_step(dtype, form, name):
    return {"few": 2.0 ** -18, "tma": 2.0 ** -11, "mma": ref.half_step(ref.DT[dtype])}["mma" if form == "general" else name]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("batch", [([1, 1], "few"), ([9, 2], "few"), ([40, 3], "tma"), ([300, 2], "tma")])
@pytest.mark.parametrize("gap", [14.3, 20.3, 24.3, 28.3])
def test_small_weights_keep_their_share(ctx, form, batch, dtype, gap):
    """A first token whose weight is 2^gap times each other's, with values of 0, over 160000 keys of equal values: the output is
    what the others' weights add up to.  A weight is off by a half step of what holds it, or 2^-31 of the largest (half of
    the smallest step, 2^-24, where the largest is 2^6); sums of equal terms in 32 bits lose up to 2^-24 a step, over at most 160000 / 16 steps."""
    new, name = batch
    length, page, d, dt = 160000, 64, 64, ref.DT[dtype]
    cu = [0, new[0], sum(new)]
    lens = [length, 5000]
    blocks = length // page
    q = torch.ones(sum(new), 2, d, dtype=dt)
    kc = torch.zeros(blocks, page, 1, d, dtype=torch.uint8)
    vc = torch.full_like(kc, pa8.code(112.0))
    kc[0, 0] = pa8.code(64.0)
    vc[0, 0] = 0
    scales = torch.ones(blocks, 1)
    scale = gap * math.log(2.0) / (64.0 * d)
    table = torch.arange(blocks, dtype=torch.int32).repeat(2, 1)
    out, lse = ctx.paged_attention_fp8(q.cuda(), kc.cuda(), vc.cuda(), scales.cuda(), scales.cuda(), table.cuda(), pa8.i32(cu), pa8.i32(lens),
                                       scale=scale, want_lse=True)
    served_by(ctx, form, name)
    u, step = ref.half_step(dt), weight_step(dtype, form, name)
    for r in range(2):
        seen = torch.arange(lens[r] - new[r] + 1, lens[r] + 1).double()[:, None, None]
        small = (seen - 1) * 2.0 ** -gap
        want = 112.0 * small / (1.0 + small)
        rel = u + step + 2.0 ** (gap - 31) + length / 16 * 2.0 ** -24
        got = out[cu[r]:cu[r + 1]].cpu().double()
        assert ((got - want).abs() <= rel * want + ref.smallest(dt)).all(), ((got / want - 1).abs().max(), rel)
        log = torch.log1p(small[..., 0]) + gap * math.log(2.0)
        assert ((lse[cu[r]:cu[r + 1]].cpu().double() - log).abs() <= 2.0 ** -10 + 2.0 ** -20 * log).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("batch, length", [(([1], "few"), 20000), (([6], "few"), 9000), (([30], "tma"), 20000), (([300], "tma"), 9000)])
def test_errors_over_long_contexts(ctx, form, batch, length, dtype):
    """Root of the mean square error against 64 bits, relative to the outputs': of the output's rounding (a half step at most, so
    1 / sqrt(3) of it), of each weight's (half a step of what holds it, independent, so in the mean of the same share), and the
    scores' in 32 bits, which turn up in the weights: (2 d + 16) 2^-24 times sum |q k| scale at most, about a quarter of that in the mean.
    A fifth more for the spread of a sample and sums in 32 bits."""
    (new, name), d, dt = batch, 128, ref.DT[dtype]
    x = pa8.make(new, [length], 8, 4, d, dtype, seed=length, low=-8, high=-7)
    wo = pa8.want_of(x, d ** -0.5)[0]
    out, _ = pa8.run(ctx, x, scale=d ** -0.5)
    served_by(ctx, form, name)
    u, step = ref.half_step(dt), weight_step(dtype, form, name)
    size = 0.8 * 0.8 * 100 * 2.0 ** -7.5 * d * d ** -0.5  # of sum |q k| scale
    limit = 1.2 * math.sqrt(u * u / 3 + step * step / 3 + (0.25 * (2 * d + 16) * 2.0 ** -24 * size) ** 2)
    err = ((out.double() - wo).square().mean() / wo.square().mean()).sqrt().item()
    assert err <= limit, (err, limit)
