"""ar_paged_plan against a plain planner: every value equal, refusals leave the step empty."""
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


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def make(cached, new, page, spare_blocks=3, spare_cols=2, seed=0, cols=None):
    rng = random.Random(seed)
    have = [-(-c // page) for c in cached]
    need = [-(-(c + n) // page) - h for c, n, h in zip(cached, new, have)]
    ids = list(range(sum(have) + max(sum(need) + spare_blocks, 0)))
    rng.shuffle(ids)
    if cols is None:
        cols = max([h + k for h, k in zip(have, need)] or [0]) + spare_cols
    table, at = [], 0
    for h in have:
        table.append((ids[at:at + h] + [-7] * cols)[:max(cols, 0)])
        at += h
    return table, ids[at:]


def check(ctx, cached, new, page, max_tokens, table, free, pad_cols=0):
    cols = len(table[0]) if table else 0
    dev = torch.full((len(table), cols + pad_cols), -9, dtype=torch.int32, device="cuda")
    if cols:
        dev[:, :cols] = ints(table)
    view = dev[:, :cols]
    want = ref.plan(cached, new, free, page, table, max_tokens)
    p = ctx.paged_plan(ints(cached), ints(new), ints(free), ints([len(free)]), view, page, max_tokens=max_tokens)
    assert ctx.last_variant == "paged_plan"
    for name in ("cu_q", "seq_lens", "slots", "positions", "free_count", "info"):
        assert getattr(p, name).tolist() == want[name], name
    assert view.tolist() == table
    assert (dev[:, cols:] == -9).all()
    assert ctx.device_status() == 0
    return p


@pytest.mark.parametrize("requests", [0, 1, 2, 31, 33, 511, 512, 513, 1500, 8192])
@pytest.mark.parametrize("page", [1, 16, 24])
def test_plan(ctx, requests, page):
    rng = random.Random(requests * 100 + page)
    cached = [rng.choice([0, 1, page - 1, page, page + 1, rng.randint(0, 60)]) for _ in range(requests)]
    new = [rng.choice([0, 1, 1, 2, page, rng.randint(0, 40)]) for _ in range(requests)]
    table, free = make(cached, new, page)
    check(ctx, cached, new, page, sum(new) + rng.choice([0, 1, 700]), table, free, pad_cols=requests % 2)


def test_long_chunk(ctx):
    cached, new = [0, 100000, 5], [70000, 1, 0]
    table, free = make(cached, new, 64)
    check(ctx, cached, new, 64, 70001 + 300, table, free)


def test_exactly_enough(ctx):
    table, free = make([16, 3], [17, 30], 16, spare_blocks=0, spare_cols=0)
    p = check(ctx, [16, 3], [17, 30], 16, 47, table, free)
    assert p.free_count.tolist() == [0]


@pytest.mark.parametrize("want, kw", [(1, dict(spare_blocks=-1)), (2, dict(cols=2)), (3, dict(max_tokens=46))])
def test_refused_whole(ctx, want, kw):
    kw = dict(kw)
    max_tokens = kw.pop("max_tokens", 47)
    table, free = make([16, 3], [17, 30], 16, **kw)
    p = check(ctx, [16, 3], [17, 30], 16, max_tokens, table, free)
    assert p.info.tolist()[:3] == [0, 0, want]


@pytest.mark.parametrize("cached, new, count", [([5, -1], [1, 1], 3), ([5, 1], [1, -4], 3), ([5, 1], [1, 1], -1), ([5, 1], [1, 1], 4),
                                                ([5, 2 ** 31 - 1], [1, 1], 3)])
def test_bad_lengths(ctx, cached, new, count):
    table = torch.full((2, 4), 7, dtype=torch.int32, device="cuda")
    p = ctx.paged_plan(ints(cached), ints(new), ints([1, 2, 3]), ints([count]), table, 16, max_tokens=8)
    assert p.info.tolist()[:3] == [0, 0, 4]
    assert p.cu_q.tolist() == [0, 0, 0] and p.slots.tolist() == [-1] * 8 and p.positions.tolist() == [0] * 8
    assert p.seq_lens.tolist() == [max(c, 0) for c in cached] and p.free_count.tolist() == [count]
    assert (table == 7).all()


def test_captured_steps_follow_the_lengths(ctx):
    """One captured plan replayed with growing lengths and the free count handed back between replays."""
    page, requests = 8, 5
    cached, new = ints([3, 0, 8, 15, 7]), ints([1] * requests)
    table = torch.full((requests, 12), -1, dtype=torch.int32, device="cuda")
    host = [[100 + 10 * r + j for j in range(-(-c // page))] + [-1] * (12 - -(-c // page)) for r, c in enumerate(cached.tolist())]
    table.copy_(ints(host))
    free, count = ints(list(range(40))), ints([40])
    out = dict(cu_q=ints([0] * 6), seq_lens=ints([0] * 5), slots=ints([0] * 8, torch.int64), positions=ints([0] * 8),
               free_count_out=ints([0]), info=ints([0] * 4))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ctx.paged_plan(cached, new, free, count, table, page, stream=s, **out)
    left, lens = list(range(40)), cached.tolist()
    for _ in range(20):
        want = ref.plan(lens, [1] * requests, left, page, host, 8)
        g.replay()
        torch.cuda.synchronize()
        assert out["slots"].tolist() == want["slots"] and table.tolist() == host and out["info"].tolist() == want["info"]
        lens, left = want["seq_lens"], left[:want["free_count"][0]]
        cached.copy_(out["seq_lens"])
        count.copy_(out["free_count_out"])


def test_binding_refuses(ctx):
    t = torch.zeros(2, 4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        ctx.paged_plan(ints([1, 1]), ints([1, 1]), ints([1]), ints([1]), t, 16)                       # no length
    with pytest.raises(ValueError):
        ctx.paged_plan(ints([1, 1]), ints([1]), ints([1]), ints([1]), t, 16, max_tokens=4)             # lengths differ
    with pytest.raises(ValueError):
        ctx.paged_plan(ints([1, 1]).cpu(), ints([1, 1]), ints([1]), ints([1]), t, 16, max_tokens=4)    # host tensor
    with pytest.raises(ValueError):
        ctx.paged_plan(ints([1, 1]).long(), ints([1, 1]), ints([1]), ints([1]), t, 16, max_tokens=4)   # type
    with pytest.raises(ValueError):
        ctx.paged_plan(ints([1, 1]), ints([1, 1]), ints([1]), ints([1]), t.t(), 16, max_tokens=4)      # table shape
