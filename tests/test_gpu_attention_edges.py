"""Calls of the attention block that its documentation allows at the edges: shared position rows, pages
released behind a window, wide caps, bad block numbers, orders in memory, many streams."""
import pytest
import torch

import serve_ref as ref
import test_gpu_paged_attention as pa
import test_gpu_qk_norm_rope as nr

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ctx():
    import tensor_all_reduce_gb300 as tar
    with tar.Context(0) as c:
        yield c


@pytest.mark.parametrize("tokens", [1, 2, 700])
@pytest.mark.parametrize("dealt", [False, True])
@pytest.mark.parametrize("d, pairs", [(128, False), (80, True), (33, False)])
def test_positions_that_all_axes_share(ctx, tokens, dealt, d, pairs):
    """Text tokens on several axes: one row expanded, against the 64-bit form and the rows written out."""
    rot = d // 2 * 2
    x = nr.make(tokens, 4, 2, d, "bf16", rot, far=1 << 20, seed=tokens)
    sections = nr.cut(rot // 2, 3)
    g = nr.on_gpu(x)
    row = g["pos"][0].clone()
    call = lambda pos: ctx.qk_norm_rope(g["q"], g["k"], None, pos, g["freq"], q_weight=g["wq"], k_weight=g["wk"], pairs=pairs,  # noqa: E731
                                        sections=sections, dealt=dealt)
    got, whole = call(row.expand(3, tokens)), call(row.repeat(3, 1))
    apart = torch.full((3, tokens + 5), -1, dtype=torch.int32, device="cuda")[:, 2:2 + tokens]
    apart.copy_(row.expand(3, tokens))
    strided = call(apart)
    axis = [0] * (rot // 2)
    for i, (n, w) in enumerate((("q", "wq"), ("k", "wk"))):
        nr.near(got[i], *ref.rope(x[n], x[w], 1e-6, False, x["pos"], x["freq"], pairs, axis))
        assert torch.equal(got[i], whole[i]) and torch.equal(got[i], strided[i])
    assert ctx.device_status() == 0


@pytest.mark.parametrize("d", [64, 128, 256])
def test_many_items_a_span(ctx, d):
    """Each CTA walks over many items, of one and two halves in turn, with rows of a warp missing: every role keeps
    the same place in the sequence, so repeated calls give equal bits, and each row is its own request's."""
    new = [1, 45, 3, 128, 0, 7, 33, 2] * 40
    lens = [(37 * i) % 290 + n for i, n in enumerate(new)]
    x = pa.make(new, lens, 6, 2, d, seed=d)
    want = pa.check(ctx, x)
    for _ in range(10):
        out, lse = pa.run(ctx, x, scale=d ** -0.5)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.fixture(params=[0, 4], ids=["auto", "general"])
def form(ctx, request):
    import tensor_all_reduce_gb300 as tar
    ctx.set_option(tar.AR_OPT_FORCE_VARIANT, request.param)
    yield request.param
    ctx.set_option(tar.AR_OPT_FORCE_VARIANT, 0)


@pytest.mark.parametrize("page", [1, 8, 16, 24, 384])
@pytest.mark.parametrize("prefix", [0, 70])
@pytest.mark.parametrize("causal", [True, False])
def test_blocks_released_behind_the_window(ctx, form, page, prefix, causal):
    """A server gives a block back as soon as no row sees a key of it (-1 in the table), inside a tile too: the
    call is right and leaves no code.  One block more is missed."""
    window, new, lens = 100, [1, 4, 300, 1], [1900, 700, 1300, 90]
    x = pa.make(new, lens, 4, 2, 64, page=page, seed=page, garbage=0.0)
    kw = dict(window=window, causal=causal)
    if prefix:
        kw["prefix_lens"] = torch.full((4,), prefix, dtype=torch.int32)
    edges = []
    for row, n, length in zip(x["table"], new, lens):
        low = max(length - n - window + 1, 0)  # the first key of the first row's window
        first, last = -(-prefix // page), low // page
        for j in range(first, last):
            row[j] = -1 if j % 2 else x["kc"].shape[0] + j
        edges.append(last)
    pa.check(ctx, x, **kw)
    for r in range(3):
        y = dict(x, table=[list(t) for t in x["table"]])
        y["table"][r][edges[r]] = -1
        pa.run(ctx, y, **kw)
        assert ctx.device_status() == 2


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("cap", [64.0, 65.0, 200.0, 1e3, 1e4, 1e6, 1e20, 1e30, 3e38, 1.0, 1e-3, 1e-30, 1e-38, 1e-42])
def test_caps_of_any_size(ctx, form, cap, d):
    """A cap costs a score no more than its own precision: with a wide one the call is the call without.
    The bound is the one of serve_ref with the cap left out: a score's error is relative to min(sum |q k| scale, cap),
    plus 2^-21 cap for caps of up to 64 (of the difference that gives the tanh; 2^-22 and its half again for log2 units)."""
    import math
    for peak in (1.0, 20.0):
        x = pa.make([1, 40], [300, 700], 2, 1, d, seed=d, garbage=0.0, peak=peak)
        scale, u = d ** -0.5, ref.half_step(torch.bfloat16)
        out, lse = pa.run(ctx, x, scale=scale, softcap=cap)
        assert ctx.device_status() == 0
        for r, (lo, hi, length) in enumerate(((0, 1, 300), (1, 41, 700))):
            blocks = torch.tensor(x["table"][r][: -(-length // 16)])
            k, v = (c[blocks].flatten(0, 1)[:length, 0].double() for c in (x["kc"], x["vc"]))
            pos, j = torch.arange(length - (hi - lo), length)[:, None], torch.arange(length)
            for h in range(2):
                q = x["q"][lo:hi, h].double()
                s = cap * torch.tanh(q @ k.t() * scale / cap)
                size = (q.abs() @ k.t().abs() * scale).clamp(max=2 * cap)
                s = s.masked_fill(j > pos, -math.inf)
                p = torch.softmax(s, -1)
                ds = (2 * d + 16) * 2.0 ** -24 * size.amax(-1, keepdim=True) + (2.0 ** -21 * cap if cap <= 64 else 0.0)
                rel = 4 * ds + 2.0 ** -20 + length * 2.0 ** -22
                want = p @ v
                eo = u * want.abs() + (1 + u) * (u + rel) * (p @ v.abs()) + ref.smallest(torch.bfloat16) * (1 + v.abs().sum(0))
                wl = torch.logsumexp(s, -1)
                el = 2 * ds[:, 0] + 2.0 ** -20 + length * 2.0 ** -22 + 2.0 ** -22 * wl.abs()
                assert ((out[lo:hi, h].double() - want).abs() <= eo).all(), (cap, peak, ((out[lo:hi, h].double() - want).abs() - eo).max())
                assert ((lse[lo:hi, h].double() - wl).abs() <= el).all(), (cap, peak, ((lse[lo:hi, h].double() - wl).abs() - el).max())


@pytest.mark.parametrize("cap", [0.0, 5.0, 1e6])
@pytest.mark.parametrize("scale", [1e38, -3e38, 1e-38])
def test_scales_of_any_size(ctx, form, scale, cap):
    """Products of 0 stay 0 whatever they are scaled by: equal weights."""
    x = pa.make([3, 30], [50, 300], 2, 1, 64, seed=3, garbage=0.0)
    x["q"].zero_()
    pa.check(ctx, x, scale=scale, softcap=cap)


@pytest.mark.parametrize("page", [1, 8])
def test_negative_block_numbers_are_no_padding(ctx, page):
    """A block number of -1 in the part of the table that is in use, or in the free list, times the page and with the
    last place of a page, is the -1 of a row without a token: the plan says -2, and both calls leave code 2."""
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cached, new = [page - 1, 0, 2 * page - 1], [1, 2 * page, 1]
    # the plan takes blocks off the end of the free list: request 0 needs one where the page is 1
    table = i32([[-1, -9, -9], [-9, -9, -9], [0, 1, -9]])
    free = i32([2, 3, -1, 4])
    p = ctx.paged_plan(i32(cached), i32(new), free, i32([4]), table, page, max_tokens=sum(new) + 2)
    assert ctx.device_status() == 2
    if page == 1:  # taken: 4 (request 0), -1 and 3 (request 1), 2 (request 2)
        want, bad = [4, -2, 3, 2], [1]
    else:          # request 0 writes the last place of its block -1; request 1 takes 4 and -1
        want, bad = [-2] + list(range(32, 40)) + [-2] * 8 + [15], [0] + list(range(9, 17))
    assert p.slots.tolist() == want + [-1, -1]
    n = len(want) + 2
    g = nr.on_gpu(nr.make(n, 4, 2, 64, "bf16", 64, page=page))
    kc = torch.full((8, page, 2, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    ctx.qk_norm_rope(g["q"], g["k"], g["v"], p.positions, g["freq"], k_cache=kc, v_cache=vc, slots=p.slots)
    assert ctx.device_status() == 2
    flat = vc.flatten(0, 1)
    for t, s in enumerate(want):
        if t not in bad:
            assert torch.equal(flat[s], g["v"][t])
            flat[s] = 3.0
    assert (flat == 3.0).all()


@pytest.mark.parametrize("order", ["block, token, which, head", "block, token, head, which", "block, head, token, which", "block, head, which, token"])
def test_keys_and_values_of_one_cache_tensor(ctx, form, order):
    """Both calls on a cache tensor whose keys and values lie between each other: as on two tensors."""
    x = pa.make([5, 1, 70], [300, 129, 70], 4, 2, 64, seed=14, garbage=0.0)
    blocks, page, hk, d = x["kc"].shape
    size = dict(block=blocks, token=page, head=hk, which=2)
    names = order.split(", ")
    one = torch.zeros([size[n] for n in names] + [d], dtype=torch.bfloat16, device="cuda")
    turned = one.permute(*[names.index(n) for n in ("which", "block", "token", "head")], 4)
    kc, vc = turned[0], turned[1]
    kc.copy_(x["kc"].cuda())
    vc.copy_(x["vc"].cuda())
    g = nr.on_gpu(nr.make(90, 4, 2, 64, "bf16", 64, page=page, seed=2))
    used = {b for t, n in zip(x["table"], x["lens"]) for b in t[: -(-n // page)]}
    slots = torch.full((90,), -1, dtype=torch.int64, device="cuda")
    rest = torch.tensor([b for b in range(blocks) if b not in used][:3], device="cuda")
    slots[: 3 * page] = (rest[:, None] * page + torch.arange(page, device="cuda")).flatten()
    two = x["kc"].cuda(), x["vc"].cuda()
    for k, v in ((kc, vc), two):
        ctx.qk_norm_rope(g["q"], g["k"], g["v"], g["pos"][0], g["freq"], q_weight=g["wq"], k_weight=g["wk"], k_cache=k, v_cache=v, slots=slots)
    assert torch.equal(kc, two[0]) and torch.equal(vc, two[1])
    a = (pa.i32(x["table"]), pa.i32(x["cu"]), pa.i32(x["lens"]))
    got, _ = ctx.paged_attention(x["q"].cuda(), kc, vc, *a)
    want, _ = ctx.paged_attention(x["q"].cuda(), *two, *a)
    assert torch.equal(got, want) and ctx.device_status() == 0


@pytest.mark.parametrize("tokens", [1, 50, 900])
def test_in_place_on_heads_of_three_parts(ctx, form, tokens):
    """q, k and v side by side in each head of the projection, q and k in place."""
    g = torch.Generator().manual_seed(tokens)
    qkv = torch.randn(tokens, 8, 3, 80, generator=g).to(torch.float16).cuda()
    y = nr.on_gpu(nr.make(tokens, 8, 8, 80, "fp16", 80, seed=1))
    q, k, v = (qkv[:, :, i] for i in range(3))
    args = dict(q_weight=y["wq"], k_weight=y["wk"], pairs=True)
    want = ctx.qk_norm_rope(q.contiguous(), k.contiguous(), None, y["pos"][0], y["freq"], **args)
    before = v.clone()
    ctx.qk_norm_rope(q, k, v, y["pos"][0], y["freq"], q_out=q, k_out=k, **args)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, before)


def test_workspaces_of_many_streams(ctx):
    """Calls on more streams than workspaces are kept for, in turn and all at once: each result as alone, and the
    memory held stays bounded."""
    ctx.release_workspaces()
    streams = [torch.cuda.Stream() for _ in range(12)]
    xs = [pa.make([1, 30], [2000 + 100 * i, 500], 6, 2, 128, seed=50 + i, garbage=0.0) for i in range(12)]
    args = [(x["q"].cuda(), x["kc"].cuda(), x["vc"].cuda(), pa.i32(x["table"]), pa.i32(x["cu"]), pa.i32(x["lens"])) for x in xs]
    want = [ctx.paged_attention(*a)[0] for a in args]
    torch.cuda.synchronize()
    ctx.release_workspaces()
    size = ctx.paged_attention_workspace(128, torch.bfloat16).numel()
    assert size < 41e6
    held = torch.cuda.memory_allocated()
    outs = [torch.empty_like(w) for w in want]
    for _ in range(10):
        for s, a, out in zip(streams, args, outs):
            ctx.paged_attention(*a, out=out, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    assert torch.cuda.memory_allocated() - held <= 8 * (size + (2 << 20)) + sum(w.numel() * 2 + 512 for w in want)
    ctx.release_workspaces()
    assert torch.cuda.memory_allocated() - held < size


@pytest.mark.parametrize("tokens, heads", [(1, 4), (5, 1), (1, 1)])
def test_single_rows_with_odd_strides(ctx, tokens, heads):
    """The stride of a dimension of one element says nothing: the aligned forms serve, with the bits of contiguous tensors."""
    def odd(t):  # the tensor with a stride of 12345 in dimensions of one element
        strides = [12345 if t.shape[i] == 1 else s for i, s in enumerate(t.stride())]
        return torch.as_strided(t, t.shape, strides)
    g = nr.on_gpu(nr.make(tokens, heads, heads, 64, "bf16", 64, seed=1))
    q, k, v = (g[x].contiguous() for x in "qkv")
    caches = [torch.zeros(1, 16, heads, 64, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    slots = torch.arange(tokens, device="cuda") + 3
    call = lambda f, kc, vc, qo: ctx.qk_norm_rope(f(q), f(k), f(v), g["pos"][0], g["freq"], q_weight=g["wq"], k_weight=g["wk"],  # noqa: E731
                                                  k_cache=f(kc), v_cache=f(vc), slots=slots, q_out=f(qo))
    want, kw = call(lambda t: t, *caches[:2], torch.empty_like(q))
    got, kg = call(odd, *caches[2:], torch.empty_like(q))
    assert ctx.last_variant == "qk_norm_rope_vec"
    assert torch.equal(got, want) and torch.equal(kg, kw) and torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    a = (pa.i32([[0]]), pa.i32([0, tokens]), pa.i32([tokens + 3]))
    want, wl = ctx.paged_attention(want, *caches[:2], *a, want_lse=True)
    got, lse = ctx.paged_attention(odd(got), odd(caches[2]), odd(caches[3]), *a, want_lse=True, out=odd(torch.empty_like(got)))
    assert ctx.last_variant == "paged_attention_tma"
    assert torch.equal(got, want) and torch.equal(lse, wl) and ctx.device_status() == 0
