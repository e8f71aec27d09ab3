"""The attention block between two fused calls, as a serving loop runs it: plan, norm and rotation with
the cache write, attention, over several steps of growing requests, eagerly and from one captured graph."""
import math

import pytest
import torch

import serve_ref as ref

pytestmark = pytest.mark.gpu

HQ, HK, D, PAGE, HIDDEN = 12, 2, 128, 16, 1536


class Loop:
    """A small layer with N = 2 partials and its request state on the GPU."""

    def __init__(self, ctx, requests, max_tokens, blocks=64, cols=24, seed=0):
        g = torch.Generator().manual_seed(seed)
        bf = torch.bfloat16
        rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.ctx, self.requests, self.max_tokens = ctx, requests, max_tokens
        self.wqkv = (rand(HIDDEN, (HQ + 2 * HK) * D) / math.sqrt(HIDDEN)).to(bf).cuda()
        self.wo = [(rand(HQ * D // 2, HIDDEN) / math.sqrt(HQ * D)).to(bf).cuda() for _ in range(2)]
        self.norm = (rand(HIDDEN) * 0.1 + 1).to(bf).cuda()
        self.qw, self.kw = ((rand(D) * 0.1 + 1).to(bf).cuda() for _ in range(2))
        self.freq = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) / (D // 2))).float().cuda()
        self.kc, self.vc = (torch.full((blocks, PAGE, HK, D), float("nan"), dtype=bf, device="cuda") for _ in range(2))
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.table, self.cached, self.new = i32(requests, cols) - 1, i32(requests), i32(requests)
        self.free = torch.randperm(blocks, generator=g).to(torch.int32).cuda()
        self.count, self.count2 = torch.tensor([blocks], dtype=torch.int32, device="cuda"), i32(1)
        self.x = [torch.zeros(max_tokens, HIDDEN, dtype=bf, device="cuda") for _ in range(2)]  # the partials of the call before
        self.res = torch.zeros(max_tokens, HIDDEN, dtype=bf, device="cuda")
        self.work = ctx.paged_attention_workspace(D, bf)

    def step(self):
        c = self.ctx
        plan = c.paged_plan(self.cached, self.new, self.free, self.count, self.table, PAGE, max_tokens=self.max_tokens, free_count_out=self.count2)
        y, res, _, _ = c.fused_reduce_rmsnorm(self.x, self.res, self.norm)
        qkv = (y @ self.wqkv).unflatten(1, (HQ + 2 * HK, D))
        q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HK], qkv[:, HQ + HK:]
        raw = qkv.clone()
        c.qk_norm_rope(q, k, v, plan.positions, self.freq, q_weight=self.qw, k_weight=self.kw, k_cache=self.kc, v_cache=self.vc,
                       slots=plan.slots, q_out=q, want_k_out=False)
        out = torch.zeros(self.max_tokens, HQ, D, dtype=torch.bfloat16, device="cuda")
        out, lse = c.paged_attention(q, self.kc, self.vc, plan.block_table, plan.cu_q, plan.seq_lens, out=out, want_lse=True, workspace=self.work)
        flat = out.flatten(1)
        partials = [flat[:, i * HQ * D // 2:(i + 1) * HQ * D // 2] @ self.wo[i] for i in range(2)]
        y2, res2, _, _ = c.fused_reduce_rmsnorm(partials, res, self.norm)
        self.cached.copy_(plan.seq_lens)
        self.count.copy_(self.count2)
        return plan, raw, q, out, lse, y2, res2


@pytest.fixture(scope="module")
def ctx():
    import tensor_all_reduce_gb300 as tar
    with tar.Context(0) as c:
        yield c


STEPS = [[20, 3, 0, 1, 40], [1, 1, 7, 1, 1], [1, 1, 1, 0, 1], [17, 1, 1, 5, 1]]


def check_step(loop, plan, raw, q, out, history, new):
    """Against the formula in 64 bits, on the kernels' own inputs to each call; `history` holds each request's
    expected k and v, as rounded by the kernel."""
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    assert plan.cu_q.tolist() == cu and plan.info.tolist()[2] == 0
    lens = [len(h) + n for h, n in zip(history, new)]
    assert plan.seq_lens.tolist() == lens
    pos, slots, table = plan.positions.cpu(), plan.slots.tolist(), plan.block_table.tolist()
    raw = raw.cpu()
    for first, w, got in ((0, loop.qw, q), (HQ, loop.kw, None)):
        heads = raw[:, first:first + (HQ if first == 0 else HK)]
        want, bound = ref.rope(heads, w.cpu(), 1e-6, False, pos[None], loop.freq.cpu(), False, [0] * (D // 2))
        if got is not None:
            assert ((got.cpu().double() - want).abs() <= bound)[:cu[-1]].all()
        else:
            kc, vc = loop.kc.cpu().flatten(0, 1), loop.vc.cpu().flatten(0, 1)
            for t in range(cu[-1]):
                assert ((kc[slots[t]].double() - want[t]).abs() <= bound[t]).all()
                assert torch.equal(vc[slots[t]], raw[t, HQ + HK:])
    assert all(s == -1 for s in slots[cu[-1]:])
    # every token's slot is its request's own, and earlier ones have not moved
    for r, h in enumerate(history):
        for t in range(cu[r], cu[r + 1]):
            h.append(slots[t])
        assert [table[r][j // PAGE] * PAGE + j % PAGE for j in range(len(h))] == h
    used = [s for h in history for s in h]
    assert len(set(used)) == len(used)
    wo, _, eo, _ = ref.attention(q.cpu(), loop.kc.cpu(), loop.vc.cpu(), table, cu, lens, D ** -0.5)
    assert ((out.cpu().double() - wo).abs() <= eo)[:cu[-1]].all() and (out[cu[-1]:] == 0).all()


def run(ctx, captured):
    loop = Loop(ctx, 5, 80)
    g = torch.Generator().manual_seed(3)
    history = [[] for _ in range(5)]
    graph = outs = None
    finals = []
    for step, new in enumerate(STEPS):
        loop.new.copy_(torch.tensor(new, dtype=torch.int32))
        for x in loop.x:
            x.copy_(torch.randn(loop.max_tokens, HIDDEN, generator=g).to(torch.bfloat16))
        if not captured:
            outs = loop.step()
        else:
            if graph is None:
                keep = [t.clone() for t in (loop.cached, loop.count, loop.table, loop.kc, loop.vc)]
                s = torch.cuda.Stream()
                s.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(s):
                    loop.step()  # warm-up: cuBLAS sets itself up
                torch.cuda.current_stream().wait_stream(s)
                torch.cuda.synchronize()
                for t, old in zip((loop.cached, loop.count, loop.table, loop.kc, loop.vc), keep):
                    t.copy_(old)
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    outs = loop.step()
            graph.replay()
        torch.cuda.synchronize()
        assert ctx.device_status() == 0
        plan, raw, q, out, lse, y2, res2 = outs
        check_step(loop, plan, raw, q, out, history, new)
        n = sum(new)
        assert torch.isfinite(y2[:n]).all() and torch.isfinite(res2[:n]).all()
        finals.append((out[:n].clone(), y2[:n].clone()))
    return finals


def test_steps_eager_and_captured(ctx):
    a, b = run(ctx, False), run(ctx, True)
    for (x, y), (u, v) in zip(a, b):
        assert torch.equal(x, u) and torch.equal(y, v)


def test_a_refused_step_changes_nothing(ctx):
    """Without blocks for the step the plan is empty, and the calls behind it leave cache and outputs alone."""
    loop = Loop(ctx, 3, 64, blocks=2)
    loop.new.copy_(torch.tensor([16, 16, 16], dtype=torch.int32))
    plan, raw, q, out, lse, _, _ = loop.step()
    torch.cuda.synchronize()
    assert plan.info.tolist() == [0, 0, 1, 3] and loop.count.tolist() == [2] and loop.cached.tolist() == [0, 0, 0]
    assert torch.isnan(loop.kc).all() and (out == 0).all() and (loop.table == -1).all()
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
            alone.append(last[3].clone())
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
        assert torch.equal(last[i][3], alone[i])
        ctxs[i].close()
