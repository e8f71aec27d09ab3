"""The attention block over a cache held in 8 bits, as a serving loop runs it between two fused calls: plan, norm and rotation
of q, append of k and v, attention, over several steps of growing requests, eagerly and from one captured graph."""
import math

import pytest
import torch

import serve8_ref as ref8
import serve_ref as ref

pytestmark = pytest.mark.gpu

HQ, HK, D, PAGE, HIDDEN = 12, 2, 128, 16, 1536
STEPS = [[20, 3, 0, 1, 40], [1, 1, 7, 1, 1], [1, 1, 1, 0, 1], [17, 1, 1, 5, 1]]


@pytest.fixture(scope="module")
def ctx():
    import tensor_all_reduce_gb300 as tar
    with tar.Context(0) as c:
        yield c


class Loop:
    """A small layer with N = 2 partials and its request state on the GPU; keys and values in one cache tensor."""

    def __init__(self, ctx, requests, max_tokens, blocks=64, cols=24, seed=0):
        g = torch.Generator().manual_seed(seed)
        bf = torch.bfloat16
        rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.ctx, self.max_tokens = ctx, max_tokens
        self.wqkv = (rand(HIDDEN, (HQ + 2 * HK) * D) / math.sqrt(HIDDEN)).to(bf).cuda()
        self.wo = [(rand(HQ * D // 2, HIDDEN) / math.sqrt(HQ * D)).to(bf).cuda() for _ in range(2)]
        self.norm = (rand(HIDDEN) * 0.1 + 1).to(bf).cuda()
        self.qw, self.kw = ((rand(D) * 0.1 + 1).to(bf).cuda() for _ in range(2))
        self.freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().cuda()
        cache = torch.full((blocks, 2, PAGE, HK, D), 0x7f, dtype=torch.uint8, device="cuda").view(ref8.E4M3)  # NaN
        self.kc, self.vc = cache[:, 0], cache[:, 1]
        self.ks, self.vs = (torch.full((blocks, HK), float("nan"), device="cuda") for _ in range(2))
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.table, self.cached, self.new = i32(requests, cols) - 1, i32(requests), i32(requests)
        self.free = torch.randperm(blocks, generator=g).to(torch.int32).cuda()
        self.count, self.count2 = torch.tensor([blocks], dtype=torch.int32, device="cuda"), i32(1)
        self.x = [torch.zeros(max_tokens, HIDDEN, dtype=bf, device="cuda") for _ in range(2)]  # the partials of the call before
        self.res = torch.zeros(max_tokens, HIDDEN, dtype=bf, device="cuda")
        self.work = ctx.paged_attention_workspace(D, bf)

    def state(self):
        return self.cached, self.count, self.table, self.kc, self.vc, self.ks, self.vs

    def step(self):
        c = self.ctx
        plan = c.paged_plan(self.cached, self.new, self.free, self.count, self.table, PAGE, max_tokens=self.max_tokens, free_count_out=self.count2)
        y, res, _, _ = c.fused_reduce_rmsnorm(self.x, self.res, self.norm)
        qkv = (y @ self.wqkv).unflatten(1, (HQ + 2 * HK, D))
        q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HK], qkv[:, HQ + HK:]
        raw = qkv.clone()
        before = [t.clone() for t in (self.kc, self.vc, self.ks, self.vs)]
        c.qk_norm_rope(q, None, None, plan.positions, self.freq, q_weight=self.qw, q_out=q)
        c.paged_append_fp8(k, v, self.kc, self.vc, self.ks, self.vs, plan.block_table, plan.cu_q, plan.seq_lens, positions=plan.positions,
                           inv_freq=self.freq, k_weight=self.kw)
        out = torch.zeros(self.max_tokens, HQ, D, dtype=torch.bfloat16, device="cuda")
        out, lse = c.paged_attention_fp8(q, self.kc, self.vc, self.ks, self.vs, plan.block_table, plan.cu_q, plan.seq_lens, out=out, want_lse=True,
                                         workspace=self.work)
        flat = out.flatten(1)
        partials = [flat[:, i * HQ * D // 2:(i + 1) * HQ * D // 2] @ self.wo[i] for i in range(2)]
        y2, res2, _, _ = c.fused_reduce_rmsnorm(partials, res, self.norm)
        self.cached.copy_(plan.seq_lens)
        self.count.copy_(self.count2)
        return plan, raw, q, before, out, lse, y2, res2


def check_step(loop, plan, raw, q, before, out, lens, new):
    """Against the formulas in 64 bits, on the kernels' own inputs to each call."""
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    assert plan.cu_q.tolist() == cu and plan.seq_lens.tolist() == lens and plan.info.tolist()[2] == 0
    raw, pos, table, n = raw.cpu(), plan.positions.cpu(), plan.block_table.tolist(), cu[-1]
    axis = [0] * (D // 2)
    want, bound = ref.rope(raw[:, :HQ], loop.qw.cpu(), 1e-6, False, pos[None], loop.freq.cpu(), False, axis)
    assert ((q.cpu().double() - want).abs() <= bound)[:n].all()
    k, ek = ref8.turned(raw[:, HQ:HQ + HK], loop.kw.cpu(), 1e-6, False, pos[None], loop.freq.cpu(), False, axis)
    v = raw[:, HQ + HK:].double()
    codes = lambda a, b, c, d: [a.cpu().view(torch.uint8), b.cpu().view(torch.uint8), c.cpu(), d.cpu()]  # noqa: E731
    after = codes(loop.kc, loop.vc, loop.ks, loop.vs)
    old = codes(*before)
    used = {b for r, x in enumerate(lens) for b in table[r][: -(-x // PAGE)]}
    rest = [b for b in range(old[2].shape[0]) if b not in used]
    for a, b in zip(old, after):  # NaN scales of blocks that nobody has
        assert torch.equal(a[rest].nan_to_num(1.0) if a.dtype.is_floating_point else a[rest], b[rest].nan_to_num(1.0) if b.dtype.is_floating_point else b[rest])
    for a in (*old[2:], *after[2:]):
        a[rest] = 1.0
    ref8.check_append(old, after, k, v, ek, torch.zeros_like(v), table, cu, lens, PAGE)
    wo, _, eo, _ = ref8.attention(q.cpu(), *after, table, cu, lens, D ** -0.5)
    assert ((out.cpu().double() - wo).abs() <= eo)[:n].all() and (out[n:] == 0).all()


def run(ctx, captured):
    loop = Loop(ctx, 5, 80)
    g = torch.Generator().manual_seed(3)
    lens = [0] * 5
    graph = outs = None
    finals = []
    for new in STEPS:
        loop.new.copy_(torch.tensor(new, dtype=torch.int32))
        for x in loop.x:
            x.copy_(torch.randn(loop.max_tokens, HIDDEN, generator=g).to(torch.bfloat16))
        if not captured:
            outs = loop.step()
        else:
            if graph is None:
                keep = [t.clone() for t in loop.state()]
                s = torch.cuda.Stream()
                s.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(s):
                    loop.step()  # warm-up: cuBLAS sets itself up
                torch.cuda.current_stream().wait_stream(s)
                torch.cuda.synchronize()
                for t, old in zip(loop.state(), keep):
                    t.copy_(old)
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    outs = loop.step()
            graph.replay()
        torch.cuda.synchronize()
        assert ctx.device_status() == 0
        plan, raw, q, before, out, lse, y2, res2 = outs
        lens = [x + n for x, n in zip(lens, new)]
        check_step(loop, plan, raw, q, before, out, lens, new)
        n = sum(new)
        assert torch.isfinite(y2[:n]).all() and torch.isfinite(res2[:n]).all()
        finals.append((out[:n].clone(), y2[:n].clone(), loop.kc.view(torch.uint8).clone(), loop.ks.clone()))
    return finals


def test_steps_eager_and_captured(ctx):
    for a, b in zip(run(ctx, False), run(ctx, True)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
        assert torch.equal(a[3].nan_to_num(0.0), b[3].nan_to_num(0.0))


def test_a_refused_step_changes_nothing(ctx):
    """Without blocks for the step the plan is empty, and the calls behind it leave cache, scales and outputs alone."""
    loop = Loop(ctx, 3, 64, blocks=2)
    loop.new.copy_(torch.tensor([16, 16, 16], dtype=torch.int32))
    plan, raw, q, before, out, lse, _, _ = loop.step()
    torch.cuda.synchronize()
    assert plan.info.tolist() == [0, 0, 1, 3] and loop.count.tolist() == [2] and loop.cached.tolist() == [0, 0, 0]
    assert (loop.kc.view(torch.uint8) == 0x7f).all() and loop.ks.isnan().all() and loop.vs.isnan().all() and (out == 0).all()
    assert ctx.device_status() == 0


def test_two_contexts_on_two_streams():
    """Two loops with contexts and streams of their own, interleaved: each as if alone."""
    import tensor_all_reduce_gb300 as tar
    alone = []
    for seed in (1, 2):
        with tar.Context(0) as c:
            loop = Loop(c, 5, 80, seed=seed)
            loop.new.copy_(torch.tensor(STEPS[0], dtype=torch.int32))
            for x in loop.x:
                x.fill_(0.5 + seed)
            for _ in range(4):
                last = loop.step()
            alone.append(last[4].clone())
            torch.cuda.synchronize()
    ctxs = [tar.Context(0) for _ in range(2)]
    loops = [Loop(c, 5, 80, seed=s) for c, s in zip(ctxs, (1, 2))]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for loop, seed in zip(loops, (1, 2)):
        loop.new.copy_(torch.tensor(STEPS[0], dtype=torch.int32))
        for x in loop.x:
            x.fill_(0.5 + seed)
    torch.cuda.synchronize()
    last = [None, None]
    for _ in range(4):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                last[i] = loops[i].step()
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(last[i][4], alone[i])
        ctxs[i].close()


def test_as_near_as_the_codes_allow(ctx):
    """Prompts appended to an 8-bit cache and attended over, against attention over the unrounded keys and values: off by what
    E4M3 keeps (half a step, 2^-4 relative, an element), averaged over the weights."""
    g = torch.Generator().manual_seed(5)
    n, hq, hk, d, page = 300, 4, 2, 64, 16
    q, k, v = (torch.randn(n, h, d, generator=g).to(torch.bfloat16) for h in (hq, hk, hk))
    blocks = -(-n // page)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    kc, vc = (torch.zeros(blocks, page, hk, d, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(blocks, hk, device="cuda") for _ in range(2))
    table, cu, lens = i32([list(range(blocks))]), i32([0, n]), i32([n])
    ctx.paged_append_fp8(k.cuda(), v.cuda(), kc, vc, ks, vs, table, cu, lens)
    out, _ = ctx.paged_attention_fp8(q.cuda(), kc, vc, ks, vs, table, cu, lens)
    pad = torch.zeros(blocks * page - n, hk, d, dtype=torch.bfloat16)
    wide = [torch.cat([x, pad]).view(blocks, page, hk, d) for x in (k, v)]
    want, _, _, _ = ref.attention(q, *wide, [list(range(blocks))], [0, n], [n], d ** -0.5)
    # values: 2^-4 of each at most; scores: 2^-4 sum |q k| scale at most, a weight by as much relative, twice (its sum)
    for h in range(hq):
        kk, vv = k[:, h // 2].double(), v[:, h // 2].double()
        s = (q[:, h].double() @ kk.t() * d ** -0.5).masked_fill(torch.arange(n) > torch.arange(n)[:, None], -math.inf)
        p = torch.softmax(s, -1)
        ds = 2.0 ** -4 * (q[:, h].double().abs() @ kk.abs().t()) * d ** -0.5
        size = torch.where(torch.isfinite(s), ds, 0.0).amax(-1, keepdim=True)
        bound = (2.0 ** -4 + torch.expm1(2 * size) * (1 + 2.0 ** -4) + 2.0 ** -7) * (p @ vv.abs())
        assert ((out[:, h].cpu().double() - want[:, h]).abs() <= bound).all()
