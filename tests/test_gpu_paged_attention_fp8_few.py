"""ar_paged_attention_fp8 for few rows a request (items of 8 and of 16 rows, requests that fill several): masks, caps, bias, scales and
queries of any size, growing maxima, NaN, blocks that are gone, many items a span."""
import pytest
import torch

import test_gpu_paged_attention_fp8 as pa8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    import tensor_all_reduce_gb300 as tar
    with tar.Context(0) as c:
        yield c


# new tokens and lengths of requests; 4 and 2 heads: up to 8 rows a request on average, up to 16
SMALL = [1, 2, 3, 1], [500, 300, 130, 1]
LARGE = [1, 7, 20, 0, 2], [700, 300, 130, 0, 2]


def check(ctx, x, **kw):
    got = pa8.check(ctx, x, **kw)
    assert ctx.last_variant == "paged_attention_fp8_few"
    return got


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [16, 64, 80, 128, 144, 256])
@pytest.mark.parametrize("new, lens", [SMALL, LARGE])
def test_masks(ctx, d, dtype, new, lens):
    x = pa8.make(new, lens, 4, 2, d, dtype, seed=d)
    check(ctx, x)
    check(ctx, x, causal=False)
    for window in (1, 17, 128, 129):
        check(ctx, x, window=window)
    pre = torch.tensor([min(n, p) for n, p in zip(lens, (100, 0, 130, 1, 2))], dtype=torch.int32)
    check(ctx, x, prefix_lens=pre)
    check(ctx, x, prefix_lens=pre, window=20)
    check(ctx, x, prefix_lens=pre, causal=False, window=5)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("new, lens", [SMALL, LARGE])
def test_cap_bias_and_scales(ctx, dtype, new, lens):
    x = pa8.make(new, lens, 4, 2, 128, dtype, seed=5, peak=4.0)
    slopes = torch.tensor([0.5, 0.25, 0.0, 1.5])
    for cap in (5.0, 50.0, 1000.0):
        check(ctx, x, softcap=cap)
    check(ctx, x, slopes=slopes)
    check(ctx, x, softcap=50.0, slopes=slopes, window=100)
    check(ctx, x, causal=False, slopes=slopes)
    for scale in (0.0, -0.3, 1.0):
        check(ctx, x, scale=scale)


@pytest.mark.parametrize("page", [8, 24, 64, 128, 384])
@pytest.mark.parametrize("hq, hk", [(1, 1), (6, 1), (8, 8), (16, 1), (48, 8), (3, 3)])
def test_heads_and_pages(ctx, page, hq, hk):
    new = [1, 1, 2, 0] if hq // hk <= 8 else [1, 1, 1, 1]
    check(ctx, pa8.make(new, [777, 128, 129, 40], hq, hk, 64, page=page, seed=page + hq))


@pytest.mark.parametrize("low, high", [(-20, 20), (-32, -28), (20, 32), (-32, 32)])
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("new, lens", [SMALL, LARGE])
def test_scales_of_any_size(ctx, low, high, d, new, lens):
    for dtype in ("bf16", "fp16"):
        x = pa8.make(new, lens, 4, 2, d, dtype, seed=6, low=low, high=high)
        x["ks"].fill_(2.0 ** -7)
        if dtype == "fp16" and high > 0:  # outputs of up to 448 * 2^high do not fit
            x["vs"] *= 2.0 ** (-high)
            x["vs"].clamp_(min=2.0 ** -32)
        check(ctx, x)
        x["ks"].fill_(2.0 ** 30)
        check(ctx, x, scale=2.0 ** -46)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new, lens", [([1, 3], [2000, 1500]), ([9, 5], [2000, 1500])])
def test_growing_maximum(ctx, d, new, lens):
    """The running maximum rises at each tile, in small steps, in leaps up and down; v scales rise and fall with them."""
    for step in (lambda j: j / 500.0, lambda j: (3000 - j) / 500.0, lambda j: ((j // 100) * 7) % 11 * 8.0):
        x = pa8.make(new, lens, 2, 1, d, seed=7, garbage=0, even=True)
        for r, length in enumerate(x["lens"]):
            for j in range(0, length, 16):
                b = x["table"][r][j // 16]
                x["kc"][b] = pa8.code(step(j))
                x["ks"][b] = 2.0 ** -3
                x["vs"][b] = 2.0 ** ((j // 16 * 5) % 31 - 15)
        x["q"] = torch.ones_like(x["q"])
        check(ctx, x, scale=4.0 / d)


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_queries_of_any_size(ctx, d, dtype):
    x = pa8.make([3, 1], [90, 300], 4, 2, d, dtype, seed=9)
    span = torch.exp2(torch.randint(-12, 13, x["q"].shape, generator=torch.Generator().manual_seed(1)).float())
    x["q"] = (x["q"].float() * span).to(x["q"].dtype)
    check(ctx, x, scale=2.0 ** -10)
    x["q"] = torch.full_like(x["q"], 65504.0 if dtype == "fp16" else 2.0 ** 100)
    check(ctx, x, scale=2.0 ** -25 if dtype == "fp16" else 2.0 ** -110)
    x["q"] = torch.full_like(x["q"], torch.finfo(x["q"].dtype).tiny)
    check(ctx, x, scale=2.0 ** 8 if dtype == "fp16" else 2.0 ** 100)
    x["q"].zero_()
    check(ctx, x)


def test_nan_reaches_the_rows_that_see_it(ctx):
    for d, ctx_len, dtype in ((64, 40, "bf16"), (64, 5000, "fp16"), (256, 700, "bf16")):
        x = pa8.make([7], [ctx_len + 7], 4, 2, d, dtype, seed=20)
        want, wl = pa8.run(ctx, x, scale=d ** -0.5)
        assert ctx.last_variant == "paged_attention_fp8_few" and torch.isfinite(want).all()
        x["q"][3, 1, d - 1] = float("nan")  # token 3, head 1
        x["q"][5, 0, 2] = float("inf")
        at = ctx_len + 4  # its place; seen by rows 4 to 6, key head 1 (heads 2 and 3)
        x["kc"][x["table"][0][at // 16], at % 16, 1, 0] = pa8.NAN_CODE
        out, lse = pa8.run(ctx, x, scale=d ** -0.5)
        bad = torch.zeros(7, 4, dtype=torch.bool)
        bad[3, 1] = bad[5, 0] = True
        bad[4:, 2:] = True
        assert out[bad].isnan().all() and lse[bad].isnan().all()
        assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse[~bad], wl[~bad])


@pytest.mark.parametrize("page", [8, 16, 24, 384])
@pytest.mark.parametrize("prefix", [0, 70])
def test_blocks_released_behind_the_window(ctx, page, prefix):
    window, new, lens = 100, [1, 4, 6, 1], [1900, 700, 1300, 90]
    x = pa8.make(new, lens, 4, 2, 64, page=page, seed=page)
    kw = dict(window=window)
    if prefix:
        kw["prefix_lens"] = torch.full((4,), prefix, dtype=torch.int32)
    spare = next(b for b in range(x["kc"].shape[0]) if not any(b in t for t in x["table"]))
    x["ks"][spare], x["vs"][spare] = float("inf"), float("nan")
    x["vc"][spare] = 0x33
    for row, n, length in zip(x["table"], new, lens):
        low = max(length - n - window + 1, 0)
        for j in range(-(-prefix // page), low // page):
            row[j] = (-1, x["kc"].shape[0] + j, spare)[j % 3]
    check(ctx, x, **kw)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("most", [2, 9])
def test_many_items_a_span(ctx, d, most):
    """Each CTA walks over many items: repeated calls give equal bits, and each row is its own request's."""
    new = [1 + i % most for i in range(600)]
    lens = [(37 * i) % 290 + n for i, n in enumerate(new)]
    x = pa8.make(new, lens, 6, 2, d, "fp16" if most > 2 else "bf16", seed=d)
    want = check(ctx, x)
    for _ in range(10):
        out, lse = pa8.run(ctx, x, scale=d ** -0.5)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_rows_that_see_nothing_and_waits(ctx):
    check(ctx, pa8.make([5, 3, 1], [2, 0, 1], 4, 2, 64))
    check(ctx, pa8.make([0, 1, 0], [50, 0, 3], 4, 2, 64, spare_rows=4), window=2)
