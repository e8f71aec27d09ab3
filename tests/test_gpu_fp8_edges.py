"""ar_paged_attention_fp8 where a product of 0 is easily lost: NaN codes in blocks that no row sees."""
import pytest
import torch

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
