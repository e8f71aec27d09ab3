"""ar_paged_attention against the formula in 64 bits: lengths from none to long, odd sizes, pages that end
inside a tile, masks that leave rows empty, splits over SMs, both kernel forms."""
import random

import pytest
import torch

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


def make(new, lens, hq, hk, d, dtype="bf16", page=16, seed=0, spare_rows=0, spare_cols=1, garbage=float("nan"), peak=1.0):
    """Inputs on the CPU.  What no request holds in the cache is `garbage`."""
    g = torch.Generator().manual_seed(seed)
    rng = random.Random(seed)
    t = ref.DT[dtype]
    need = [-(-x // page) for x in lens]
    blocks = sum(need) + 3
    ids = list(range(blocks))
    rng.shuffle(ids)
    cols = max(need + [0]) + spare_cols
    kc = torch.full((blocks * page, hk, d), garbage, dtype=t)
    vc = kc.clone()
    table, at = [], 0
    for x, n in zip(lens, need):
        row = ids[at:at + n]
        at += n
        if x:
            j = torch.arange(x)
            slot = torch.tensor(row)[j // page] * page + j % page
            kc[slot] = torch.randn(x, hk, d, generator=g).to(t)
            vc[slot] = torch.randn(x, hk, d, generator=g).to(t)
        table.append(row + [-1] * (cols - n))
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = (torch.randn(cu[-1] + spare_rows, hq, d, generator=g) * peak).to(t)
    return dict(q=q, kc=kc.view(blocks, page, hk, d), vc=vc.view(blocks, page, hk, d), table=table, cu=cu, lens=lens)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def run(ctx, x, **kw):
    q = x["q"].cuda()
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device="cuda")
    table = i32(x["table"]) if x["table"] else torch.zeros(0, 1, dtype=torch.int32, device="cuda")
    gpu = {n: v.cuda() if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    ctx.paged_attention(q, x["kc"].cuda(), x["vc"].cuda(), table, i32(x["cu"]), i32(x["lens"]), out=out, lse=lse, **gpu)
    torch.cuda.synchronize()
    return out.cpu(), lse.cpu()


def check(ctx, x, scale=None, **kw):
    d = x["q"].shape[-1]
    scale = d ** -0.5 if scale is None else scale
    named = dict(kw)
    if "prefix_lens" in named:
        named["prefix"] = named.pop("prefix_lens").tolist()
    wo, wl, eo, el = ref.attention(x["q"], x["kc"], x["vc"], x["table"], x["cu"], x["lens"], scale, **named)
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
@pytest.mark.parametrize("d", [64, 80, 96, 128, 256, 8, 72, 200, 33, 1])
def test_head_sizes(ctx, form, dtype, d):
    check(ctx, make([1, 20, 0, 7], [50, 20, 9, 300], 6, 2, d, dtype, seed=d))


@pytest.mark.parametrize("page", [1, 5, 8, 16, 24, 32, 48, 64, 128, 256, 384])
def test_page_sizes(ctx, form, page):
    check(ctx, make([1, 33, 130], [700, 400, 130], 4, 2, 64, page=page, seed=page))


@pytest.mark.parametrize("hq, hk", [(1, 1), (12, 2), (6, 1), (8, 8), (7, 1), (40, 8), (20, 4), (64, 1), (300, 1)])
def test_head_groups(ctx, form, hq, hk):
    check(ctx, make([3, 1, 40], [3, 260, 100], hq, hk, 64, seed=hq))


@pytest.mark.parametrize("length", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000, 4097])
def test_single_token_lengths(ctx, form, length):
    check(ctx, make([1], [length], 12, 2, 128, seed=length))


@pytest.mark.parametrize("n", [2, 10, 11, 21, 22, 42, 43, 63, 64, 65, 128, 129, 200, 257])
def test_chunk_lengths(ctx, form, n):
    check(ctx, make([n], [n + 37], 6, 1, 128, seed=n))
    check(ctx, make([n], [n], 3, 3, 64, seed=n))


def test_empty_calls(ctx, form):
    check(ctx, make([0, 0], [0, 9], 4, 2, 64, spare_rows=5))
    check(ctx, make([0, 0, 2, 0], [0, 9, 2, 0], 4, 2, 64, spare_rows=5))
    x = make([], [], 4, 2, 64, spare_rows=3)
    out, lse = run(ctx, x)
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


def test_cap_and_bias(ctx, form):
    x = make([30, 1], [200, 700], 4, 2, 128, seed=5, peak=4.0)
    slopes = torch.tensor([0.5, 0.25, 0.0, 1.5])
    check(ctx, x, softcap=5.0)
    check(ctx, x, slopes=slopes)
    check(ctx, x, softcap=50.0, slopes=slopes, window=100, prefix_lens=torch.tensor([64, 3], dtype=torch.int32))
    check(ctx, x, causal=False, slopes=slopes)


def test_scales(ctx, form):
    x = make([30, 1], [200, 700], 4, 2, 128, seed=6)
    check(ctx, x, scale=0.0)
    check(ctx, x, scale=-0.3)
    check(ctx, x, scale=1.0)     # one key takes nearly all


def test_growing_maximum(ctx, form):
    """Later keys score higher and higher, so the running maximum rises at each tile; and the reverse."""
    for sign in (1.0, -1.0):
        x = make([5, 200], [2000, 1500], 2, 1, 64, seed=7, garbage=0.0)
        for r, length in enumerate(x["lens"]):
            for j in range(length):
                x["kc"][x["table"][r][j // 16], j % 16] = (sign * j / 60.0) / 8.0
        x["q"] = torch.ones_like(x["q"])
        check(ctx, x)
    for d in (128, 256):  # in leaps of more than the 2^8 that the reference tolerates, up and down
        x = make([5, 150], [1500, 1500], 2, 1, d, seed=d, garbage=0.0)
        for r, length in enumerate(x["lens"]):
            for j in range(length):
                x["kc"][x["table"][r][j // 16], j % 16] = (((j // 100) * 7) % 11) * 16.0 / d
        x["q"] = torch.ones_like(x["q"])
        check(ctx, x, scale=1.0)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_items_of_one_and_two_halves(ctx, form, d):
    """Requests of few and of many rows in turn, one tile of keys and many, in one CTA's span and over several."""
    new = [1, 90, 2, 60, 1, 1, 130, 43, 42, 1, 0, 200, 3]
    lens = [5, 90, 900, 61, 300, 129, 140, 43, 2000, 128, 77, 1000, 3]
    check(ctx, make(new * 2, lens * 2, 6, 2, d, seed=d))
    check(ctx, make(new * 12, [min(x, 300) for x in lens] * 12, 15, 5, d, "fp16", seed=d + 1))


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
    x = make([2, 5], [200, 90], 4, 2, 64, seed=19, garbage=0.0)
    x["table"][1][:4] = x["table"][0][:4]
    x["table"][0][7] = x["table"][0][6]
    check(ctx, x)


def test_long_cache_is_split(ctx, form):
    """One token over 20000 keys: the keys are shared out over the SMs and joined."""
    x = make([1], [20000], 4, 1, 128, seed=9)
    a = check(ctx, x)
    b = run(ctx, x, scale=128 ** -0.5)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])  # the same bits


def test_infinities_where_nothing_is_seen(ctx, form):
    for bad in (float("inf"), float("-inf"), float("nan")):
        check(ctx, make([20, 1], [100, 77], 4, 2, 64, seed=10, garbage=bad, page=32))


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
    ctx.paged_attention(x["q"].cuda(), x["kc"].cuda(), x["vc"].cuda(), i32(x["table"]), i32(x["cu"]), i32(x["lens"]), scale=d ** -0.5,
                        out=out, workspace=room_w[2 * shift:][:work.numel()])
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), want)
    assert (room[:, :shift] == 7.0).all() and (room[:, shift + 6 * d:] == 7.0).all()


def test_nan_reaches_the_rows_that_see_it(ctx, form):
    """A NaN in a query or a visible key: its rows are NaN, every other row keeps its bits."""
    for d, ctx_len in ((64, 40), (64, 5000), (256, 700)):
        x = make([70], [ctx_len + 70], 4, 2, d, seed=20)
        want, wl = run(ctx, x, scale=d ** -0.5)
        assert torch.isfinite(want).all()
        x["q"][3, 1, d - 1] = float("nan")  # token 3, head 1
        at = ctx_len + 60  # its place; seen by rows 60 to 69, key head 1 (heads 2 and 3)
        page = x["kc"].shape[1]
        x["kc"][x["table"][0][at // page], at % page, 1, 0] = float("nan")
        out, lse = run(ctx, x, scale=d ** -0.5)
        bad = torch.zeros(70, 4, dtype=torch.bool)
        bad[3, 1] = True
        bad[60:, 2:] = True
        bad = bad.to(out.device)
        assert out[bad].isnan().all() and lse[bad].isnan().all()
        assert torch.equal(out[~bad], want[~bad]) and torch.equal(lse[~bad], wl[~bad])


def test_keys_outside_the_window_may_be_gone(ctx, form):
    """Blocks that lie before every row's window are not read: their numbers may be anything."""
    x = make([1, 4], [900, 700], 4, 2, 64, seed=11)
    for row, n in zip(x["table"], (900 - 100, 700 - 103)):
        for j in range(n // 128 * 8):  # whole tiles before the window
            row[j] = -1
    check(ctx, x, window=100)


def test_bad_block_numbers_read_as_zeros(ctx, form):
    x = make([2, 1], [200, 50], 4, 2, 64, seed=12, garbage=0.0)
    blocks = x["kc"].shape[0]
    x["table"][0][3], x["table"][0][5], x["table"][1][0] = blocks, -5, 1 << 30
    out, lse = run(ctx, x, scale=0.125)
    assert ctx.device_status() == 2
    zero = dict(x, kc=torch.cat([x["kc"], torch.zeros_like(x["kc"][:1])]), vc=torch.cat([x["vc"], torch.zeros_like(x["vc"][:1])]))
    zero["table"] = [list(t) for t in x["table"]]
    zero["table"][0][3] = zero["table"][0][5] = zero["table"][1][0] = blocks
    wo, wl, eo, el = ref.attention(zero["q"], zero["kc"], zero["vc"], zero["table"], zero["cu"], zero["lens"], 0.125)
    assert ((out.double() - wo).abs() <= eo).all() and ((lse.double() - wl).abs() <= el).all()


def test_lengths_beyond_the_table_are_cut(ctx, form):
    x = make([2, 1], [64, 48], 4, 2, 64, seed=13, spare_cols=0)
    wo, wl, eo, el = ref.attention(x["q"], x["kc"], x["vc"], x["table"][:1], x["cu"][:2], [64], 0.125)
    x["lens"] = [1000000, 48]
    out, _ = run(ctx, x, scale=0.125)
    assert ctx.device_status() == 2
    assert ((out.double() - wo).abs()[:2] <= eo[:2]).all()
    x["lens"], x["cu"] = [64, -3], [0, 2, 9]  # a negative length, rows behind the end
    out, _ = run(ctx, x, scale=0.125)
    assert ctx.device_status() == 2
    assert ((out.double() - wo).abs()[:2] <= eo[:2]).all() and (out[2] == 0).all()


def test_orders_and_strides(ctx, form):
    x = make([5, 1, 70], [300, 129, 70], 4, 2, 64, seed=14, garbage=0.0)
    want, wl = check(ctx, x)
    kc, vc, q = x["kc"].cuda(), x["vc"].cuda(), x["q"].cuda()
    both = torch.stack([kc, vc], 1).transpose(2, 3).contiguous().transpose(2, 3)  # [block, k or v, head, token, dim] in memory
    wide = torch.zeros(q.shape[0], 4, 3, 64, dtype=q.dtype, device="cuda")
    wide[:, :, 1] = q
    cols = len(x["table"][0])
    table = torch.full((3, 100), -1, dtype=torch.int32, device="cuda")
    table[:, :cols] = i32(x["table"])
    out = torch.zeros(q.shape[0], 4 * 64 + 8, dtype=q.dtype, device="cuda")[:, :256].unflatten(1, (4, 64))
    ctx.paged_attention(wide[:, :, 1], both[:, 0], both[:, 1], table[:, :cols], i32(x["cu"]), i32(x["lens"]), out=out)
    assert torch.equal(out.cpu(), want)
    # off a 16-byte boundary
    buf = torch.zeros(kc.numel() + 1, dtype=kc.dtype, device="cuda")
    odd = buf[1:].view(kc.shape)
    odd.copy_(kc)
    got, _ = ctx.paged_attention(q, odd, vc, table[:, :cols], i32(x["cu"]), i32(x["lens"]))
    wo, _, eo, _ = ref.attention(x["q"], x["kc"], x["vc"], x["table"], x["cu"], x["lens"], 0.125)
    assert ((got.cpu().double() - wo).abs() <= eo).all()


def test_captured_call_follows_the_lengths(ctx, form):
    """Captured once, replayed with other lengths and tables; a second graph with its own workspace beside it."""
    x = make([1, 1, 1], [700, 300, 90], 6, 2, 128, seed=15, garbage=0.0)
    q, kc, vc, table, cu, lens = x["q"].cuda(), x["kc"].cuda(), x["vc"].cuda(), i32(x["table"]), i32(x["cu"]), i32(x["lens"])
    graphs, outs = [], []
    for _ in range(2):
        s = torch.cuda.Stream()
        out = torch.zeros_like(q)
        ws = ctx.paged_attention_workspace(128, q.dtype)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            ctx.paged_attention(q, kc, vc, table, cu, lens, out=out, workspace=ws, stream=s)
        graphs.append((g, s, ws))
        outs.append(out)
    for new_lens in ([700, 300, 90], [1, 16, 17], [512, 299, 3]):
        lens.copy_(i32(new_lens))
        torch.cuda.synchronize()
        for _ in range(5):
            for g, s, _ws in graphs:
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        wo, _, eo, _ = ref.attention(x["q"], x["kc"], x["vc"], x["table"], x["cu"], new_lens, 128 ** -0.5)
        for out in outs:
            assert ((out.cpu().double() - wo).abs() <= eo).all()


def test_own_workspaces(ctx):
    """Without a workspace: calls on two streams at once, and a captured call replayed beside eager ones, each
    have their own."""
    xs = [make([1, 1], [3000 + 500 * i, 700], 6, 2, 128, seed=30 + i, garbage=0.0) for i in range(3)]
    args = [(x["q"].cuda(), x["kc"].cuda(), x["vc"].cuda(), i32(x["table"]), i32(x["cu"]), i32(x["lens"])) for x in xs]
    want = [ctx.paged_attention(*a)[0].clone() for a in args]
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    out = torch.zeros_like(args[2][0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ctx.paged_attention(*args[2], out=out)
    for _ in range(20):
        a = ctx.paged_attention(*args[0], stream=s)[0]
        with torch.cuda.stream(t):
            b = ctx.paged_attention(*args[1])[0]
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(out, want[2])
        out.zero_()


def test_offsets_beyond_32_bits(ctx, form):
    """A cache of more than 2^32 elements: the last blocks are read at their own place."""
    page, hk, d = 64, 8, 128
    blocks = (1 << 32) // (page * hk * d) + 200
    kc = torch.zeros(blocks, page, hk, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    small = make([3], [200], 16, 8, d, page=page, seed=16, garbage=0.0)
    table = [[blocks - 1 - b for b in small["table"][0][:4]]]
    for far, close in zip(table[0], small["table"][0]):
        kc[far], vc[far] = small["kc"][close].cuda(), small["vc"][close].cuda()
    out, _ = ctx.paged_attention(small["q"].cuda(), kc, vc, i32(table), i32(small["cu"]), i32(small["lens"]))
    wo, _, eo, _ = ref.attention(small["q"], small["kc"], small["vc"], small["table"], small["cu"], small["lens"], d ** -0.5)
    assert ((out.cpu().double() - wo).abs() <= eo).all()


def test_a_wait_that_runs_out_ends_the_call(ctx):
    """The first copy of each CTA is held back: the call ends with code 1, and the next one is right."""
    import tensor_all_reduce_gb300 as tar
    x = make([40, 1], [500, 3000], 4, 2, 128, seed=17, garbage=0.0)
    ctx.set_option(tar.AR_OPT_TEST_STALL, 1)
    ctx.set_option(tar.AR_OPT_WAIT_CYCLES, 2000000)
    try:
        run(ctx, x)
        assert ctx.last_variant == "paged_attention_tma"
        assert ctx.device_status() == 1
    finally:
        ctx.set_option(tar.AR_OPT_TEST_STALL, 0)
        ctx.set_option(tar.AR_OPT_WAIT_CYCLES, 0)
    check(ctx, x)


def test_forms(ctx):
    """Which form serves which call."""
    import tensor_all_reduce_gb300 as tar
    for d, page, want in ((128, 16, "tma"), (64, 128, "tma"), (80, 24, "tma"), (256, 16, "tma"), (128, 4, "mma"), (36, 16, "mma"), (256, 7, "mma")):
        check(ctx, make([3], [50], 4, 2, d, page=page))
        assert ctx.last_variant == "paged_attention_" + want
    ctx.set_option(tar.AR_OPT_FORCE_VARIANT, 4)
    check(ctx, make([3], [50], 4, 2, 128))
    assert ctx.last_variant == "paged_attention_mma"
    ctx.set_option(tar.AR_OPT_FORCE_VARIANT, 0)


def test_binding_refuses(ctx):
    x = make([2], [20], 4, 2, 64)
    q, kc, vc, t, cu, lens = x["q"].cuda(), x["kc"].cuda(), x["vc"].cuda(), i32(x["table"]), i32(x["cu"]), i32(x["lens"])
    import tensor_all_reduce_gb300 as tar
    for bad in (lambda: ctx.paged_attention(q.float(), kc, vc, t, cu, lens), lambda: ctx.paged_attention(q, kc.half(), vc, t, cu, lens),
                lambda: ctx.paged_attention(q[:, :3], kc, vc, t, cu, lens), lambda: ctx.paged_attention(q, kc, vc[:2], t, cu, lens),
                lambda: ctx.paged_attention(q, kc, vc, t, cu[:1], lens), lambda: ctx.paged_attention(q, kc, vc, t.long(), cu, lens),
                lambda: ctx.paged_attention(q.cpu(), kc, vc, t, cu, lens)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(tar.ArError):
        ctx.paged_attention(q, kc, vc, t, cu, lens, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(tar.ArError):
        ctx.paged_attention(q, kc, vc, t, cu, lens, out=q)
    with pytest.raises(tar.ArError):
        ctx.paged_attention(q, kc, vc, t, cu, lens, window=-1)
