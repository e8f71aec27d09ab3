"""Which arrays of the attention block's calls share bytes, without a GPU: layouts that lie between each other are
taken (AR_ERR_NOT_INITIALIZED: the arguments are right), ones that meet are refused; and a check of the rule against
sets of bytes."""
import random

import pytest

import tensor_all_reduce_gb300 as tar
import test_serve_host as host
from test_serve_host import D, HK, HQ, NI, OV, at, lib  # noqa: F401

B, P = 10, 16  # blocks of a cache, tokens of a block


def cache(k, v, ks, vs):
    """The strides of block, token and head of two caches, in elements, and their addresses."""
    return dict(k_cache=at(7) + 2 * k, v_cache=at(7) + 2 * v, k_block_stride=ks[0], k_page_stride=ks[1], k_cache_head_stride=ks[2],
                v_block_stride=vs[0], v_page_stride=vs[1], v_cache_head_stride=vs[2], num_blocks=B, page_size=P)


@pytest.mark.parametrize("want, kw", [
    (NI, cache(0, P * HK * D, (2 * P * HK * D, HK * D, D), (2 * P * HK * D, HK * D, D))),          # [block, k or v, token, head, dim]
    (NI, cache(0, HK * D, (2 * P * HK * D, 2 * HK * D, D), (2 * P * HK * D, 2 * HK * D, D))),      # [block, token, k or v, head, dim]
    (NI, cache(0, D, (2 * P * HK * D, 2 * HK * D, 2 * D), (2 * P * HK * D, 2 * HK * D, 2 * D))),   # [block, token, head, k or v, dim]
    (NI, cache(D, 0, (2 * P * HK * D, 2 * HK * D, 2 * D), (2 * P * HK * D, 2 * HK * D, 2 * D))),   # v before k
    (NI, cache(0, D, (2 * P * HK * D, 2 * D, 2 * P * D), (2 * P * HK * D, 2 * D, 2 * P * D))),     # [block, head, token, k or v, dim]
    (NI, cache(0, P * D, (2 * P * HK * D, D, 2 * P * D), (2 * P * HK * D, D, 2 * P * D))),         # [block, head, k or v, token, dim]
    (NI, cache(0, B * P * HK * D, (P * HK * D, HK * D, D), (P * HK * D, HK * D, D))),              # [k or v, block, ...]
    (OV, cache(0, D - 1, (2 * P * HK * D, 2 * HK * D, 2 * D), (2 * P * HK * D, 2 * HK * D, 2 * D))),
    (OV, cache(0, HK * D - D, (2 * P * HK * D, 2 * HK * D, D), (2 * P * HK * D, 2 * HK * D, D))),
    (OV, cache(0, D, (2 * P * HK * D, 2 * HK * D, D), (2 * P * HK * D, 2 * HK * D, 2 * D))),
    (OV, cache(0, D, (2 * P * HK * D + D, 2 * HK * D, 2 * D), (2 * P * HK * D + D, 2 * HK * D, 2 * D))),
])
def test_caches(want, kw):
    assert host.rope(**kw) == want


def packed(order, **kw):
    """q, k and v of as many heads as views of one projection [token, head, 3, dim] (or another order), q and k in place."""
    h = 4
    step = {"head": D, "three": h * D}[order]
    ts, hs = 3 * h * D, {"head": 3 * D, "three": D}[order]
    q, k, v = (at(0) + 2 * i * step for i in range(3))
    d = dict(q_heads=h, kv_heads=h, q=q, k=k, v=v, q_out=q, k_out=k, q_token_stride=ts, k_token_stride=ts, v_token_stride=ts, q_head_stride=hs,
             k_head_stride=hs, v_head_stride=hs, q_out_token_stride=ts, q_out_head_stride=hs, k_out_token_stride=ts, k_out_head_stride=hs,
             k_cache=None, v_cache=None)
    d.update(kw)
    return d


@pytest.mark.parametrize("want, kw", [
    (NI, packed("head")), (NI, packed("head", tokens=1, q_heads=1, kv_heads=4, q=at(0), q_out=at(0))), (NI, packed("three")), (NI, packed("head", tokens=1)), (NI, packed("head", tokens=0)),
    (OV, packed("head", k_out=at(0))), (OV, packed("head", k_out=at(0) + 2 * (D + 8))), (OV, packed("three", q_out=at(0) + 2 * D)),
    (OV, packed("head", q_out_head_stride=3 * D + 8)), (OV, packed("head", tokens=1, k_out=at(0) + 2 * (D + 8))),
])
def test_packed_projections_in_place(want, kw):
    assert host.rope(**kw) == want


def test_queries_and_outputs_of_one_tensor():
    both = dict(q_token_stride=2 * HQ * D, q_head_stride=2 * D, out=at(0) + 2 * D, out_token_stride=2 * HQ * D, out_head_stride=2 * D)
    assert host.attention(**both) == NI
    assert host.attention(**dict(both, out=at(0) + 2 * D - 2)) == OV


def test_the_rule_never_passes_arrays_that_meet():
    """Random small arrays of q_out against k: whatever the call takes shares no byte."""
    rng = random.Random(5)
    taken = 0
    for _ in range(4000):
        n, h, g, d = rng.randint(1, 4), rng.randint(1, 3), rng.randint(1, 3), rng.choice([1, 2, 4])
        hs, ks = (rng.choice([d, d + 1, 2 * d, 3 * d, 12]) for _ in range(2))
        ts, kt = (rng.choice([d, 2 * d, 3 * hs, 12, 24, 36, 5]) for _ in range(2))
        off = rng.randint(0, 40)
        st = host.rope(tokens=n, q_heads=h, kv_heads=g, head_dim=d, rot_dim=0, positions=None, inv_freq=None, q_weight=None, k_weight=None,
                       k_cache=None, v_cache=None, q=at(1), q_token_stride=h * d, q_head_stride=d, q_out=at(0), q_out_token_stride=ts, q_out_head_stride=hs,
                       k=at(0) + 2 * off, k_token_stride=kt, k_head_stride=ks, k_out=at(2), k_out_token_stride=g * d, k_out_head_stride=d)
        if st != NI:
            assert st in (OV, tar.AR_ERR_INVALID_ARG)
            continue
        taken += 1
        a = {t * ts + x * hs + e for t in range(n) for x in range(h) for e in range(d)}
        b = {off + t * kt + x * ks + e for t in range(n) for x in range(g) for e in range(d)}
        assert not a & b, (n, h, g, d, hs, ks, ts, kt, off)
    assert taken > 300


@pytest.mark.parametrize("want, heads, cols", [(NI, 64, 1 << 26), (tar.AR_ERR_UNSUPPORTED, 65, 1 << 26), (tar.AR_ERR_UNSUPPORTED, 65536, 1 << 20),
                                               (NI, 65536, 1 << 16), (NI, 8, (1 << 31) - 1)])
def test_tiles_that_32_bits_count(want, heads, cols):
    """Tables that name more key tiles over all heads than the division of the work counts are refused."""
    far = 1 << 44  # the other operands, away from so long a table and cache
    kw = dict(q_heads=heads, kv_heads=heads, head_dim=8, tokens=4, requests=1, table_cols=cols, page_size=16, num_blocks=1,
              q_token_stride=heads * 8, q_head_stride=8, out_token_stride=heads * 8, out_head_stride=8, k_block_stride=128 * heads, k_page_stride=8 * heads,
              k_head_stride=8, v_block_stride=128 * heads, v_page_stride=8 * heads, v_head_stride=8, block_table=far, workspace=2 * far)
    assert host.attention(**kw) == want
