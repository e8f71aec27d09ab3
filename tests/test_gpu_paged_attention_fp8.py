"""ar_paged_attention_fp8 against the formula in 64 bits: lengths from none to long, odd sizes, pages that end inside
a tile, scales of any size, masks that leave rows empty, splits over SMs, both kernel forms."""
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


NAN_CODE = 0x7f


def code(value):
    return torch.tensor([value]).to(ref8.E4M3).view(torch.uint8).item()


def make(new, lens, hq, hk, d, dtype="bf16", page=16, seed=0, spare_rows=0, spare_cols=1, garbage=NAN_CODE, peak=1.0, low=-9, high=-4, even=False):
    """Inputs on the CPU.  What no request holds in the cache is the code `garbage`, its scales NaN; the others'
    scales lie between 2^low and 2^high."""
    g = torch.Generator().manual_seed(seed)
    rng = random.Random(seed)
    need = [-(-x // page) for x in lens]
    blocks = sum(need) + 3
    ids = list(range(blocks))
    rng.shuffle(ids)
    cols = max(need + [0]) + spare_cols
    c = {}
    for n in ("k", "v"):
        codes = torch.full((blocks * page, hk, d), garbage, dtype=torch.uint8)
        e = torch.rand(blocks, hk, generator=g) * (high - low) + low
        c[n + "s"] = torch.exp2(torch.round(e) if even else e)
        c[n + "c"] = codes
    table, at, used = [], 0, set()
    for x, n in zip(lens, need):
        row = ids[at:at + n]
        used.update(row)
        at += n
        if x:
            j = torch.arange(x)
            slot = torch.tensor(row)[j // page] * page + j % page
            for m in ("kc", "vc"):
                c[m][slot] = (torch.randn(x, hk, d, generator=g) * 100).clamp(-448, 448).to(ref8.E4M3).view(torch.uint8)
        table.append(row + [-1] * (cols - n))
    for n in ("ks", "vs"):
        c[n][[b for b in range(blocks) if b not in used]] = float("nan")
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = (torch.randn(cu[-1] + spare_rows, hq, d, generator=g) * peak).to(ref.DT[dtype])
    return dict(q=q, kc=c["kc"].view(blocks, page, hk, d), vc=c["vc"].view(blocks, page, hk, d), ks=c["ks"], vs=c["vs"], table=table, cu=cu, lens=lens)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def on_gpu(x):
    table = i32(x["table"]) if x["table"] else torch.zeros(0, 1, dtype=torch.int32, device="cuda")
    return (x["q"].cuda(), *(x[n].cuda() for n in ("kc", "vc", "ks", "vs")), table, i32(x["cu"]), i32(x["lens"]))


def run(ctx, x, **kw):
    a = on_gpu(x)
    out = torch.full_like(a[0], 7.0)
    lse = torch.full(a[0].shape[:2], 7.0, dtype=torch.float32, device="cuda")
    gpu = {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    ctx.paged_attention_fp8(*a, out=out, lse=lse, **gpu)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu()


def want_of(x, scale, **kw):
    return ref8.attention(x["q"], x["kc"], x["vc"], x["ks"], x["vs"], x["table"], x["cu"], x["lens"], scale, **kw)


def check(ctx, x, scale=None, **kw):
    d = x["q"].shape[-1]
    scale = d ** -0.5 if scale is None else scale
    named = dict(kw)
    if "prefix_lens" in named:
        named["prefix"] = named.pop("prefix_lens").tolist()
    wo, wl, eo, el = want_of(x, scale, **named)
    out, lse = run(ctx, x, scale=scale, **kw)
    assert ctx.device_status() == 0
    mine = torch.zeros(x["q"].shape[0], dtype=torch.bool)
    mine[x["cu"][0]:x["cu"][-1]] = True
    assert (out[~mine] == 7.0).all() and (lse[~mine] == 7.0).all()
    assert torch.isfinite(out).all()
    over = ((out.double() - wo).abs() - eo)[mine]
    assert (over <= 0).all(), f"out: {over.max().item():.3g} over a bound of {eo[mine].flatten()[over.argmax()].item():.3g}"
    empty = torch.isinf(wl)
    assert torch.equal(torch.isinf(lse) & mine[:, None], empty & mine[:, None]) and (lse[mine][empty[mine]] < 0).all()
    assert (out[mine][empty[mine]] == 0).all()
    some = mine[:, None] & ~empty
    assert ((lse.double() - wl).abs()[some] <= el[some]).all(), f"lse: {((lse.double() - wl).abs() - el)[some].max().item():.3g} over"
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 80, 96, 128, 256, 16, 208, 8, 72, 200, 33, 1])
def test_head_sizes(ctx, form, dtype, d):
    check(ctx, make([1, 20, 0, 7], [50, 20, 9, 300], 6, 2, d, dtype, seed=d))


@pytest.mark.parametrize("page", [1, 5, 8, 16, 24, 32, 48, 64, 128, 256, 384])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_page_sizes(ctx, form, page, dtype):
    check(ctx, make([1, 33, 130], [700, 400, 130], 4, 2, 64, dtype, page=page, seed=page))


@pytest.mark.parametrize("hq, hk", [(1, 1), (12, 2), (6, 1), (8, 8), (7, 1), (40, 8), (20, 4), (64, 1), (300, 1)])
def test_head_groups(ctx, form, hq, hk):
    check(ctx, make([3, 1, 40], [3, 260, 100], hq, hk, 64, seed=hq))


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000, 4097])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_single_token_lengths(ctx, form, length, dtype):
    check(ctx, make([1], [length], 12, 2, 128, dtype, seed=length))


@pytest.mark.parametrize("n", [2, 10, 11, 21, 22, 42, 43, 63, 64, 65, 128, 129, 200, 257])
def test_chunk_lengths(ctx, form, n):
    check(ctx, make([n], [n + 37], 6, 1, 128, seed=n))
    check(ctx, make([n], [n], 3, 3, 64, "fp16", seed=n))


def test_empty_calls(ctx, form):
    check(ctx, make([0, 0], [0, 9], 4, 2, 64, spare_rows=5))
    check(ctx, make([0, 0, 2, 0], [0, 9, 2, 0], 4, 2, 64, spare_rows=5))
    out, lse = run(ctx, make([], [], 4, 2, 64, spare_rows=3))
    assert (out == 7.0).all() and (lse == 7.0).all() and ctx.last_variant == "none"


def test_rows_that_see_nothing(ctx, form):
    # more new tokens than cached ones: the first rows lie before the first key
    check(ctx, make([10, 3, 5], [4, 0, 5], 4, 2, 64))
    check(ctx, make([300, 1], [4, 0], 4, 2, 64, spare_rows=2), window=2)


def test_masks(ctx, form):
    x = make([40, 1, 130], [500, 300, 130], 4, 2, 64, seed=4)
    check(ctx, x, causal=False)
    for window in (1, 2, 17, 64, 128, 129, 1 << 29, 2 ** 31 - 1):
        check(ctx, x, window=window)
        check(ctx, x, window=window, causal=False)
    pre = torch.tensor([100, 0, 130], dtype=torch.int32)
    check(ctx, x, prefix_lens=pre)
    check(ctx, x, prefix_lens=pre, window=20)
    check(ctx, x, prefix_lens=torch.tensor([1, 300, 3], dtype=torch.int32), window=1)
    check(ctx, x, prefix_lens=torch.tensor([480, 299, 64], dtype=torch.int32), causal=False, window=5)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_cap_and_bias(ctx, form, dtype):
    x = make([30, 1], [200, 700], 4, 2, 128, dtype, seed=5, peak=4.0)
    slopes = torch.tensor([0.5, 0.25, 0.0, 1.5])
    check(ctx, x, softcap=5.0)
    check(ctx, x, softcap=1000.0)
    check(ctx, x, slopes=slopes)
    check(ctx, x, softcap=50.0, slopes=slopes, window=100, prefix_lens=torch.tensor([64, 3], dtype=torch.int32))
    check(ctx, x, causal=False, slopes=slopes)


def test_scales_of_the_scores(ctx, form):
    x = make([30, 1], [200, 700], 4, 2, 128, seed=6)
    check(ctx, x, scale=0.0)
    check(ctx, x, scale=-0.3)
    check(ctx, x, scale=1.0)     # one key takes nearly all


@pytest.mark.parametrize("low, high", [(-20, 20), (-32, -28), (20, 32), (-32, 32)])
@pytest.mark.parametrize("d", [64, 256])
def test_scales_of_any_size(ctx, form, low, high, d):
    """Values of very different sizes side by side; keys are kept of one size by the scale of the scores."""
    for dtype in ("bf16", "fp16"):
        x = make([30, 1, 3], [200, 700, 90], 4, 2, d, dtype, seed=6, low=low, high=high)
        x["ks"].fill_(2.0 ** -7)
        top = 2.0 ** 9
        if dtype == "fp16" and high > 0:  # outputs of up to 448 * 2^high do not fit
            x["vs"] *= 2.0 ** (-high)
            x["vs"].clamp_(min=2.0 ** -32)
        check(ctx, x)
        x["ks"].fill_(2.0 ** 30)
        check(ctx, x, scale=2.0 ** -37 / top)


def test_scales_outside_their_range(ctx, form):
    """0, negative, tiny, huge, infinite ones and NaN count as the nearer end of the range, NaN as the lower."""
    x = make([3, 1], [100, 60], 4, 2, 64, seed=7)
    odd = [0.0, -1.0, 2.0 ** -100, float("nan"), 1e-40]
    for i, s in enumerate(odd):
        x["ks"][x["table"][0][i], i % 2] = s
        x["vs"][x["table"][0][i], 1 - i % 2] = s
    check(ctx, x)
    for s in (2.0 ** 100, float("inf")):
        x["vs"][x["table"][1][1], 1] = s
        check(ctx, x)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_one_key_over_many_small_ones(ctx, form, dtype):
    """A first token that takes most of the weight, and thousands that share the rest, whose values all point one
    way: small weights must not drown."""
    x = make([1, 3], [20000, 9000], 2, 1, 64, dtype, seed=8, garbage=0, even=True)
    x["q"].fill_(1.0)
    x["ks"].fill_(2.0 ** -7)
    x["vs"].fill_(2.0 ** -7)
    x["kc"].zero_()
    x["vc"].fill_(code(100.0))
    for first in (448.0, 200.0):
        for r in range(2):
            x["kc"][x["table"][r][0], 0] = code(first)
            x["vc"][x["table"][r][0], 0] = code(-300.0)
        for scale in (0.02, 0.05, 0.1):
            check(ctx, x, scale=scale)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_growing_maximum(ctx, form, d):
    """Later keys score higher and higher, so the running maximum rises at each tile, in small steps, in leaps up and
    down; v scales rise and fall with them."""
    for step in (lambda j: j / 500.0, lambda j: (3000 - j) / 500.0, lambda j: ((j // 100) * 7) % 11 * 8.0):
        x = make([5, 200], [2000, 1500], 2, 1, d, seed=7, garbage=0, even=True)
        for r, length in enumerate(x["lens"]):
            for j in range(0, length, 16):
                b = x["table"][r][j // 16]
                x["kc"][b] = code(step(j))
                x["ks"][b] = 2.0 ** -3
                x["vs"][b] = 2.0 ** ((j // 16 * 5) % 31 - 15)
        x["q"] = torch.ones_like(x["q"])
        check(ctx, x, scale=4.0 / d)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_queries_of_any_size(ctx, form, d, dtype):
    """Rows of very different sizes, and rows whose elements are: each keeps its own precision."""
    x = make([40, 1], [90, 300], 4, 2, d, dtype, seed=9)
    span = torch.exp2(torch.randint(-12, 13, x["q"].shape, generator=torch.Generator().manual_seed(1)).float())
    x["q"] = (x["q"].float() * span).to(x["q"].dtype)
    check(ctx, x, scale=2.0 ** -10)
    x["q"] = torch.full_like(x["q"], 65504.0 if dtype == "fp16" else 2.0 ** 100)
    check(ctx, x, scale=2.0 ** -25 if dtype == "fp16" else 2.0 ** -110)
    x["q"] = torch.full_like(x["q"], torch.finfo(x["q"].dtype).tiny)
    check(ctx, x, scale=2.0 ** 8 if dtype == "fp16" else 2.0 ** 100)
    x["q"].zero_()
    check(ctx, x)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_items_of_one_and_two_halves(ctx, form, d):
    """Requests of few and of many rows in turn, one tile of keys and many, in one CTA's span and over several."""
    new = [1, 90, 2, 60, 1, 1, 130, 43, 42, 1, 0, 200, 3]
    lens = [5, 90, 900, 61, 300, 129, 140, 43, 2000, 128, 77, 1000, 3]
    check(ctx, make(new * 2, lens * 2, 6, 2, d, seed=d))
    check(ctx, make(new * 12, [min(x, 300) for x in lens] * 12, 15, 5, d, "fp16", seed=d + 1))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_items_a_span(ctx, d):
    """Each CTA walks over many items, of one and two halves in turn, with rows of a warp missing: repeated calls give
    equal bits, and each row is its own request's."""
    new = [1, 45, 3, 128, 0, 7, 33, 2] * 40
    lens = [(37 * i) % 290 + n for i, n in enumerate(new)]
    x = make(new, lens, 6, 2, d, seed=d)
    want = check(ctx, x)
    for _ in range(10):
        out, lse = run(ctx, x, scale=d ** -0.5)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("seed", range(6))
def test_mixed_batches(ctx, form, seed):
    rng = random.Random(seed)
    r = rng.choice([3, 17, 200])
    new = [rng.choice([0, 1, 1, 1, 1, rng.randint(2, 90)]) for _ in range(r)]
    lens = [n + rng.choice([0, rng.randint(0, 900 if r < 100 else 100)]) for n in new]
    check(ctx, make(new, lens, 6, 2, rng.choice([64, 128]), rng.choice(["bf16", "fp16"]), rng.choice([8, 16, 32, 40]), seed=seed, spare_rows=rng.choice([0, 4])))


def test_many_requests(ctx, form):
    check(ctx, make([1] * 700, [1 + i % 37 for i in range(700)], 2, 1, 64, page=8, seed=8))
    new = [(1, 0, 2, 0, 0, 30)[i % 6] if i % 50 else 70 for i in range(3000)]  # several rounds of requests a CTA's threads
    check(ctx, make(new, [n + i % 41 for i, n in enumerate(new)], 2, 1, 64, page=8, seed=9))


def test_rows_that_begin_behind_the_first(ctx, form):
    """cu_q need not start at 0: the rows in front belong to nobody."""
    x = make([3, 0, 50], [40, 5, 300], 4, 2, 64, seed=18)
    x["q"] = torch.cat([x["q"][:7], x["q"]])
    x["cu"] = [c + 7 for c in x["cu"]]
    check(ctx, x)


def test_requests_that_share_blocks(ctx, form):
    """A common prefix kept once: two tables name the same blocks, also twice in one table."""
    x = make([2, 5], [200, 90], 4, 2, 64, seed=19, garbage=0)
    x["table"][1][:4] = x["table"][0][:4]
    x["table"][0][7] = x["table"][0][6]
    check(ctx, x)


def test_long_cache_is_split(ctx, form):
    """One token over 20000 keys: the keys are shared out over the SMs and joined."""
    x = make([1], [20000], 4, 1, 128, seed=9)
    a = check(ctx, x)
    b = run(ctx, x, scale=128 ** -0.5)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])  # the same bits


@pytest.mark.parametrize("shift", [0, 8])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_on_16_and_32_byte_boundaries(ctx, d, shift):
    """Outputs and workspace that begin 16 bytes behind a 32-byte boundary, rows of an odd number of 16 bytes: the same bits."""
    x = make([1, 90, 300, 2], [4000, 2100, 300, 64], 6, 2, d, seed=21)
    want, _ = run(ctx, x, scale=d ** -0.5)
    n = x["q"].shape[0]
    room = torch.full((n, 6 * d + 8 + shift), 7.0, dtype=x["q"].dtype, device="cuda")
    out = torch.as_strided(room, (n, 6, d), (6 * d + 8 + shift, d, 1), shift)
    work = ctx.paged_attention_workspace(d, x["q"].dtype)
    room_w = torch.empty(work.numel() + 16, dtype=torch.uint8, device="cuda")
    ctx.paged_attention_fp8(*on_gpu(x), scale=d ** -0.5, out=out, workspace=room_w[2 * shift:][:work.numel()])
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want)
    assert (room[:, :shift] == 7.0).all() and (room[:, shift + 6 * d:] == 7.0).all()


def test_nan_reaches_the_rows_that_see_it(ctx, form):
    """A NaN in a query or a visible key: its rows are NaN, every other row keeps its bits."""
    for d, ctx_len, dtype in ((64, 40, "bf16"), (64, 5000, "fp16"), (256, 700, "bf16"), (256, 70, "fp16")):
        x = make([70], [ctx_len + 70], 4, 2, d, dtype, seed=20)
        want, wl = run(ctx, x, scale=d ** -0.5)
        assert torch.isfinite(want).all()
        x["q"][3, 1, d - 1] = float("nan")  # token 3, head 1
        x["q"][5, 0, 2] = float("inf")
        at = ctx_len + 60  # its place; seen by rows 60 to 69, key head 1 (heads 2 and 3)
        x["kc"][x["table"][0][at // 16], at % 16, 1, 0] = NAN_CODE
        out, lse = run(ctx, x, scale=d ** -0.5)
        bad = torch.zeros(70, 4, dtype=torch.bool)
        bad[3, 1] = bad[5, 0] = True
        bad[60:, 2:] = True
        assert out[bad].isnan().all() and lse[bad].isnan().all()
        assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse[~bad], wl[~bad])


@pytest.mark.parametrize("page", [1, 8, 16, 24, 384])
@pytest.mark.parametrize("prefix", [0, 70])
@pytest.mark.parametrize("causal", [True, False])
def test_blocks_released_behind_the_window(ctx, form, page, prefix, causal):
    """A block that no row sees may be gone (-1 in the table) or another's, with scales of any kind, inside a tile too."""
    window, new, lens = 100, [1, 4, 300, 1], [1900, 700, 1300, 90]
    x = make(new, lens, 4, 2, 64, page=page, seed=page)
    kw = dict(window=window, causal=causal)
    if prefix:
        kw["prefix_lens"] = torch.full((4,), prefix, dtype=torch.int32)
    spare = next(b for b in range(x["kc"].shape[0]) if not any(b in t for t in x["table"]))  # of NaN codes...
    x["ks"][spare], x["vs"][spare] = float("inf"), float("nan")
    x["vc"][spare] = 0x33  # ...values are finite, their scale is not
    edges = []
    for row, n, length in zip(x["table"], new, lens):
        low = max(length - n - window + 1, 0)  # the first key of the first row's window
        first, last = -(-prefix // page), low // page
        for j in range(first, last):
            row[j] = (-1, x["kc"].shape[0] + j, spare)[j % 3]
        edges.append(last)
    check(ctx, x, **kw)
    for r in range(3):
        y = dict(x, table=[list(t) for t in x["table"]])
        y["table"][r][edges[r]] = -1
        run(ctx, y, **kw)
        assert ctx.device_status() == 2


def test_bad_block_numbers_read_as_zeros(ctx, form):
    x = make([2, 1], [200, 50], 4, 2, 64, seed=12, garbage=0, even=True)
    blocks = x["kc"].shape[0]
    x["table"][0][3], x["table"][0][5], x["table"][1][0] = blocks, -5, 1 << 30
    out, lse = run(ctx, x, scale=0.125)
    assert ctx.device_status() == 2
    zero = dict(x, table=[list(t) for t in x["table"]])
    for n in ("kc", "vc"):
        zero[n] = torch.cat([x[n], torch.zeros_like(x[n][:1])])
    for n in ("ks", "vs"):
        zero[n] = torch.cat([x[n], torch.ones_like(x[n][:1])])
    zero["table"][0][3] = zero["table"][0][5] = zero["table"][1][0] = blocks
    wo, wl, eo, el = want_of(zero, 0.125)
    assert ((out.double() - wo).abs() <= eo).all() and ((lse.double() - wl).abs() <= el).all()


def test_lengths_beyond_the_table_are_cut(ctx, form):
    x = make([2, 1], [64, 48], 4, 2, 64, seed=13, spare_cols=0)
    wo, wl, eo, el = want_of(dict(x, table=x["table"][:1], cu=x["cu"][:2], lens=[64]), 0.125)
    x["lens"] = [1000000, 48]
    out, _ = run(ctx, x, scale=0.125)
    assert ctx.device_status() == 2
    assert ((out.double() - wo).abs()[:2] <= eo[:2]).all()
    x["lens"], x["cu"] = [64, -3], [0, 2, 9]  # a negative length, rows behind the end
    out, _ = run(ctx, x, scale=0.125)
    assert ctx.device_status() == 2
    assert ((out.double() - wo).abs()[:2] <= eo[:2]).all() and (out[2] == 0).all()


def test_orders_and_strides(ctx, form):
    x = make([5, 1, 70], [300, 129, 70], 4, 2, 64, seed=14, garbage=0)
    want, wl = check(ctx, x)
    q, kc, vc, ks, vs, _, cu, lens = on_gpu(x)
    both = torch.stack([kc, vc], 1).transpose(2, 3).contiguous().transpose(2, 3)  # [block, k or v, head, token, dim] in memory
    wide = torch.zeros(q.shape[0], 4, 3, 64, dtype=q.dtype, device="cuda")
    wide[:, :, 1] = q
    cols = len(x["table"][0])
    table = torch.full((3, 100), -1, dtype=torch.int32, device="cuda")
    table[:, :cols] = i32(x["table"])
    out = torch.zeros(q.shape[0], 4 * 64 + 8, dtype=q.dtype, device="cuda")[:, :256].unflatten(1, (4, 64))
    scales = torch.stack([vs, ks]).permute(2, 0, 1).contiguous()  # [head, v or k, block]
    codes = both.view(torch.float8_e4m3fn)
    ctx.paged_attention_fp8(wide[:, :, 1], codes[:, 0], both[:, 1], scales[:, 1].t(), scales[:, 0].t(), table[:, :cols], cu, lens, out=out)
    assert torch.equal(out.cpu(), want)
    # one scale for all: expanded
    one = torch.full((1, 1), 2.0 ** -6, device="cuda").expand(ks.shape)
    a, _ = ctx.paged_attention_fp8(q, kc, vc, one, one, table[:, :cols], cu, lens)
    b, _ = ctx.paged_attention_fp8(q, kc, vc, one.contiguous(), one.contiguous(), table[:, :cols], cu, lens)
    assert torch.equal(a, b)
    wo, _, eo, _ = want_of(x, 0.125)
    for off in (1, 4, 8):  # off a 16-byte boundary
        buf = torch.zeros(kc.numel() + off, dtype=torch.uint8, device="cuda")
        odd = buf[off:].view(kc.shape)
        odd.copy_(kc)
        got, _ = ctx.paged_attention_fp8(q, odd, vc, ks, vs, table[:, :cols], cu, lens)
        assert ((got.cpu().double() - wo).abs() <= eo).all()


def test_captured_call_follows_the_lengths(ctx, form):
    """Captured once, replayed with other lengths and scales; a second graph with its own workspace beside it."""
    x = make([1, 1, 1], [700, 300, 90], 6, 2, 128, seed=15, garbage=0)
    a = on_gpu(x)
    graphs, outs = [], []
    for _ in range(2):
        s = torch.cuda.Stream()
        out = torch.zeros_like(a[0])
        ws = ctx.paged_attention_workspace(128, a[0].dtype)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            ctx.paged_attention_fp8(*a, out=out, workspace=ws, stream=s)
        graphs.append((g, s, ws))
        outs.append(out)
    for new_lens in ([700, 300, 90], [1, 16, 17], [512, 299, 3]):
        a[7].copy_(i32(new_lens))
        x["vs"] = x["vs"] * 1.5
        a[4].copy_(x["vs"])
        torch.cuda.synchronize()
        for _ in range(5):
            for g, s, _ws in graphs:
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        wo, _, eo, _ = want_of(dict(x, lens=new_lens), 128 ** -0.5)
        for out in outs:
            assert ((out.cpu().double() - wo).abs() <= eo).all()


def test_own_workspaces(ctx):
    """Without a workspace: calls over 8- and 16-bit caches on two streams at once, and a captured call replayed beside
    eager ones, each have their own."""
    xs = [make([1, 1], [3000 + 500 * i, 700], 6, 2, 128, seed=30 + i, garbage=0) for i in range(3)]
    args = [on_gpu(x) for x in xs]
    q, kc, vc, _, _, table, cu, lens = args[1]
    wide = (q, *(c.view(torch.float8_e4m3fn).to(torch.bfloat16) for c in (kc, vc)), table, cu, lens)
    want = [ctx.paged_attention_fp8(*a)[0].clone() for a in args] + [ctx.paged_attention(*wide)[0].clone()]
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    out = torch.zeros_like(args[2][0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ctx.paged_attention_fp8(*args[2], out=out)
    for _ in range(20):
        a = ctx.paged_attention_fp8(*args[0], stream=s)[0]
        with torch.cuda.stream(t):
            b = ctx.paged_attention_fp8(*args[1])[0]
            c = ctx.paged_attention(*wide)[0]
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(out, want[2]) and torch.equal(c, want[3])
        out.zero_()


def test_offsets_beyond_32_bits(ctx, form):
    """A cache of more than 2^32 elements: the last blocks are read at their own place."""
    page, hk, d = 64, 8, 128
    blocks = (1 << 32) // (page * hk * d) + 200
    kc = torch.zeros(blocks, page, hk, d, dtype=torch.uint8, device="cuda")
    vc = torch.zeros_like(kc)
    ks, vs = (torch.ones(blocks, hk, device="cuda") for _ in range(2))
    small = make([3], [200], 16, 8, d, page=page, seed=16, garbage=0)
    table = [[blocks - 1 - b for b in small["table"][0][:4]]]
    for far, close in zip(table[0], small["table"][0]):
        for to, n in ((kc, "kc"), (vc, "vc"), (ks, "ks"), (vs, "vs")):
            to[far] = small[n][close].cuda()
    out, _ = ctx.paged_attention_fp8(small["q"].cuda(), kc, vc, ks, vs, i32(table), i32(small["cu"]), i32(small["lens"]))
    wo, _, eo, _ = want_of(small, d ** -0.5)
    assert ((out.cpu().double() - wo).abs() <= eo).all()


def test_binding_refuses(ctx):
    import tensor_all_reduce_gb300 as tar
    q, kc, vc, ks, vs, t, cu, lens = on_gpu(make([2], [20], 4, 2, 64))
    f = ctx.paged_attention_fp8
    for bad in (lambda: f(q.float(), kc, vc, ks, vs, t, cu, lens), lambda: f(q, kc.half(), vc, ks, vs, t, cu, lens),
                lambda: f(q[:, :3], kc, vc, ks, vs, t, cu, lens), lambda: f(q, kc, vc[:2], ks, vs, t, cu, lens),
                lambda: f(q, kc, vc, ks.double(), vs, t, cu, lens), lambda: f(q, kc, vc, ks, vs[:, :1], t, cu, lens),
                lambda: f(q, kc, vc, ks[1:], vs, t, cu, lens), lambda: f(q, kc, vc, ks, vs.cpu(), t, cu, lens),
                lambda: f(q, kc.view(torch.int8), vc, ks, vs, t, cu, lens), lambda: f(q, kc, vc, ks, vs, t, cu[:1], lens)):
        with pytest.raises(ValueError):
            bad()
    for kw in (dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda")), dict(out=q), dict(window=-1)):
        with pytest.raises(tar.ArError):
            f(q, kc, vc, ks, vs, t, cu, lens, **kw)


def test_forms(ctx):
    """Which form serves which call."""
    import tensor_all_reduce_gb300 as tar
    for d, page, want in ((128, 16, "few"), (64, 128, "few"), (80, 24, "few"), (16, 8, "few"), (256, 16, "few"), (128, 4, "mma"), (72, 16, "mma"),
                          (36, 16, "mma"), (256, 7, "mma")):
        check(ctx, make([8], [50], 4, 2, d, page=page))
        assert ctx.last_variant == "paged_attention_fp8_" + want
        check(ctx, make([9], [50], 4, 2, d, page=page))
        assert ctx.last_variant == "paged_attention_fp8_" + want.replace("few", "tma")
    ctx.set_option(tar.AR_OPT_FORCE_VARIANT, 4)
    check(ctx, make([3], [50], 4, 2, 128))
    assert ctx.last_variant == "paged_attention_fp8_mma"
    ctx.set_option(tar.AR_OPT_FORCE_VARIANT, 0)


@pytest.mark.parametrize("new, form", [([40, 1], "tma"), ([300, 1], "tma"), ([1, 2], "few")])
def test_a_wait_that_runs_out_ends_the_call(ctx, new, form):
    """The first copy of each CTA is held back: the call ends with code 1, and the next one is right."""
    import tensor_all_reduce_gb300 as tar
    x = make(new, [500, 3000], 4, 2, 128, seed=17, garbage=0)
    ctx.set_option(tar.AR_OPT_TEST_STALL, 1)
    ctx.set_option(tar.AR_OPT_WAIT_CYCLES, 2000000)
    try:
        run(ctx, x)
        assert ctx.last_variant == "paged_attention_fp8_" + form
        assert ctx.device_status() == 1
    finally:
        ctx.set_option(tar.AR_OPT_TEST_STALL, 0)
        ctx.set_option(tar.AR_OPT_WAIT_CYCLES, 0)
    check(ctx, x)
