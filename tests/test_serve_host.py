"""Refusals of the attention block's entry points, without a GPU: a call whose arguments are right
returns AR_ERR_NOT_INITIALIZED with ctx = NULL, a wrong one its own error, and nothing runs."""
import ctypes

import pytest

import tensor_all_reduce_gb300 as tar

BASE, MB = 1 << 40, 1 << 20   # fake, well-aligned device addresses; never dereferenced
NI, IA, AL, OV, UN = (tar.AR_ERR_NOT_INITIALIZED, tar.AR_ERR_INVALID_ARG, tar.AR_ERR_ALIGNMENT, tar.AR_ERR_OVERLAP,
                      tar.AR_ERR_UNSUPPORTED)


def at(i):
    return BASE + i * 64 * MB


@pytest.fixture(scope="module", autouse=True)
def lib():
    from tensor_all_reduce_gb300 import _build
    _build.build()
    return tar.load_library()


def plan(**kw):
    d = dict(requests=4, page_size=16, max_tokens=100, free_capacity=50, table_cols=10, table_stride=0, cached_lens=at(0), new_lens=at(1),
             free_blocks=at(2), free_count=at(3), block_table=at(4), cu_q=at(5), seq_lens=at(6), slots=at(7), positions=at(8),
             free_count_out=at(9), info=at(10))
    d.update(kw)
    return tar.ar_paged_plan(None, tar.ArPagedPlanArgs(**d), None, raise_on_error=False)


@pytest.mark.parametrize("want, kw", [
    (NI, {}), (NI, dict(requests=0, cached_lens=None, new_lens=None, block_table=None, seq_lens=None)), (NI, dict(max_tokens=0, slots=None, positions=None)),
    (NI, dict(table_stride=64)), (NI, dict(requests=tar.AR_MAX_REQUESTS)),
    (IA, dict(requests=-1)), (IA, dict(requests=tar.AR_MAX_REQUESTS + 1)), (IA, dict(page_size=0)), (IA, dict(page_size=65537)),
    (IA, dict(max_tokens=-1)), (IA, dict(max_tokens=(1 << 30) + 1)), (IA, dict(free_capacity=-1)), (IA, dict(table_cols=-1)),
    (IA, dict(table_stride=9)), (IA, dict(cached_lens=None)), (IA, dict(new_lens=None)), (IA, dict(free_blocks=None)), (IA, dict(free_count=None)),
    (IA, dict(block_table=None)), (IA, dict(cu_q=None)), (IA, dict(slots=None)), (IA, dict(positions=None)), (IA, dict(info=None)),
    (IA, dict(free_count_out=None)), (AL, dict(slots=at(7) + 4)), (AL, dict(cu_q=at(5) + 2)),
    (OV, dict(free_count_out=at(3))), (OV, dict(seq_lens=at(0))), (OV, dict(positions=at(7) + 400)), (OV, dict(block_table=at(2))),
    (OV, dict(info=at(5) + 16)),
])
def test_plan_refusals(want, kw):
    assert plan(**kw) == want


D, T, HQ, HK = 128, 32, 12, 2


def rope(sections=(), **kw):
    row = (HQ + 2 * HK) * D
    d = dict(tokens=T, q_heads=HQ, kv_heads=HK, head_dim=D, dtype=tar.AR_DTYPE_BF16, q=at(0), k=at(0) + HQ * D * 2, v=at(0) + (HQ + HK) * D * 2,
             q_token_stride=row, q_head_stride=D, k_token_stride=row, k_head_stride=D, v_token_stride=row, v_head_stride=D, q_out=at(1), k_out=at(2),
             q_out_token_stride=HQ * D, q_out_head_stride=D, k_out_token_stride=HK * D, k_out_head_stride=D, q_weight=at(3), k_weight=at(4),
             eps=1e-6, gemma=0, rot_dim=D, pairs=0, axes=1, dealt=0, positions=at(5), position_stride=0, inv_freq=at(6), k_cache=at(7), v_cache=at(8),
             k_block_stride=16 * HK * D, k_page_stride=HK * D, k_cache_head_stride=D, v_block_stride=16 * HK * D, v_page_stride=HK * D,
             v_cache_head_stride=D, num_blocks=10, page_size=16, slots=at(9))
    d.update(kw)
    a = tar.ArQkNormRopeArgs(**d)
    for i, n in enumerate(sections):
        a.sections[i] = n
    return tar.ar_qk_norm_rope(None, a, None, raise_on_error=False)


ROW = (HQ + 2 * HK) * D


@pytest.mark.parametrize("want, kw", [
    (NI, {}), (NI, dict(tokens=0)), (NI, dict(k_out=None)), (NI, dict(k_cache=None, v_cache=None, slots=None, v=None)),
    (NI, dict(q_weight=None, k_weight=None)), (NI, dict(rot_dim=0, positions=None, inv_freq=None)), (NI, dict(q_heads=0, q=None, q_out=None)),
    (NI, dict(axes=3, sections=(20, 22, 22))), (NI, dict(axes=2, sections=(64, 0), dealt=1)),
    # in place, q and k of the packed projection at their own strides
    (NI, dict(q_out=at(0), q_out_token_stride=ROW, k_out=at(0) + HQ * D * 2, k_out_token_stride=ROW)),
    # one cache tensor [blocks, 2, page, heads, dim]
    (NI, dict(k_block_stride=32 * HK * D, v_block_stride=32 * HK * D, v_cache=at(7) + 16 * HK * D * 2)),
    (IA, dict(tokens=-1)), (IA, dict(q_heads=-1)), (IA, dict(q_heads=0, kv_heads=0)), (IA, dict(head_dim=0)), (IA, dict(head_dim=257)),
    (IA, dict(dtype=tar.AR_DTYPE_F32)), (IA, dict(eps=-1.0)), (IA, dict(eps=float("nan"))), (IA, dict(eps=float("inf"))), (IA, dict(rot_dim=63)),
    (IA, dict(rot_dim=D + 2)), (IA, dict(axes=0)), (IA, dict(axes=5)), (IA, dict(axes=3, sections=(20, 22, 21))),
    (IA, dict(axes=2, sections=(65, -1))), (IA, dict(axes=2, sections=(32, 32), position_stride=T - 1)), (IA, dict(q=None)), (IA, dict(q_out=None)),
    (IA, dict(k=None)), (IA, dict(k_out=None, k_cache=None, v_cache=None)), (IA, dict(v_cache=None)), (IA, dict(slots=None)), (IA, dict(v=None)),
    (IA, dict(positions=None)), (IA, dict(inv_freq=None)), (IA, dict(page_size=0)), (IA, dict(num_blocks=-1)), (IA, dict(q_head_stride=D - 1)),
    (IA, dict(k_token_stride=-1)), (IA, dict(k_cache_head_stride=1)),
    (AL, dict(q=at(0) + 1)), (AL, dict(q_out=at(1) + 1)), (AL, dict(slots=at(9) + 4)), (AL, dict(inv_freq=at(6) + 2)), (AL, dict(k_weight=at(4) + 1)),
    (OV, dict(q_out=at(0))),                                    # on q, at another stride
    (OV, dict(q_out=at(0) + 2, q_out_token_stride=ROW)),        # shifted by an element
    (OV, dict(k_out=at(1))), (OV, dict(v_cache=at(7))), (OV, dict(q_out=at(3))), (OV, dict(k_out=at(9))), (OV, dict(k_cache=at(5))),
    (OV, dict(k_out=at(0) + (HQ + HK) * D * 2, k_out_token_stride=ROW)),  # on v
])
def test_rope_refusals(want, kw):
    assert rope(**kw) == want


def attention(**kw):
    d = dict(tokens=T, requests=4, q_heads=HQ, kv_heads=HK, head_dim=D, dtype=tar.AR_DTYPE_BF16, q=at(0), out=at(1), q_token_stride=HQ * D,
             q_head_stride=D, out_token_stride=HQ * D, out_head_stride=D, lse=at(2), k_cache=at(3), v_cache=at(4), k_block_stride=16 * HK * D,
             k_page_stride=HK * D, k_head_stride=D, v_block_stride=16 * HK * D, v_page_stride=HK * D, v_head_stride=D, num_blocks=100, page_size=16,
             block_table=at(5), table_cols=10, table_stride=0, cu_q=at(6), seq_lens=at(7), scale=0.1, causal=1, window=0, softcap=0.0, slopes=at(8),
             prefix_lens=at(9), workspace=at(10), workspace_bytes=1 << 40)
    d.update(kw)
    return tar.ar_paged_attention(None, tar.ArPagedAttentionArgs(**d), None, raise_on_error=False)


@pytest.mark.parametrize("want, kw", [
    (NI, {}), (NI, dict(tokens=0)), (NI, dict(requests=0)), (NI, dict(lse=None, slopes=None, prefix_lens=None)), (NI, dict(window=1 << 30)),
    (NI, dict(num_blocks=0, k_cache=None, v_cache=None)), (NI, dict(softcap=30.0, causal=0)),
    (IA, dict(tokens=-1)), (IA, dict(requests=-1)), (IA, dict(requests=tar.AR_MAX_REQUESTS + 1)), (IA, dict(q_heads=13)), (IA, dict(kv_heads=0)),
    (IA, dict(head_dim=0)), (IA, dict(head_dim=257)), (IA, dict(dtype=tar.AR_DTYPE_F32)), (IA, dict(scale=float("nan"))), (IA, dict(softcap=-1.0)),
    (IA, dict(softcap=float("inf"))), (IA, dict(window=-1)), (IA, dict(page_size=0)), (IA, dict(num_blocks=-1)), (IA, dict(table_cols=-1)),
    (IA, dict(table_stride=9)), (IA, dict(q=None)), (IA, dict(out=None)), (IA, dict(k_cache=None)), (IA, dict(v_cache=None)), (IA, dict(block_table=None)),
    (IA, dict(cu_q=None)), (IA, dict(seq_lens=None)), (IA, dict(workspace=None)), (IA, dict(q_head_stride=1)), (IA, dict(out_token_stride=5)),
    (UN, dict(tokens=1 << 30)),
    (AL, dict(q=at(0) + 1)), (AL, dict(lse=at(2) + 2)), (AL, dict(workspace=at(10) + 8)), (AL, dict(block_table=at(5) + 2)),
    (OV, dict(out=at(0))), (OV, dict(out=at(3) + 64)), (OV, dict(lse=at(1))), (OV, dict(workspace=at(1))), (OV, dict(lse=at(6))),
])
def test_attention_refusals(want, kw):
    assert attention(**kw) == want


def test_workspace_query_refusals():
    n = ctypes.c_size_t()
    lib = tar.load_library()
    ask = lambda **kw: lib.ar_paged_attention_workspace(None, ctypes.byref(tar.ArPagedAttentionArgs(**kw)), ctypes.byref(n))  # noqa: E731
    assert ask(head_dim=128, dtype=tar.AR_DTYPE_BF16) == NI
    assert ask(head_dim=0, dtype=tar.AR_DTYPE_BF16) == IA
    assert ask(head_dim=300, dtype=tar.AR_DTYPE_F16) == IA
    assert ask(head_dim=128, dtype=tar.AR_DTYPE_F32) == IA
    assert lib.ar_paged_attention_workspace(None, None, ctypes.byref(n)) == IA


def test_argument_blocks_match_the_header(tmp_path):
    """Size and every offset of the argument structures, asked of a C compiler."""
    import os
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    pairs = [("ar_paged_plan_args", tar.ArPagedPlanArgs), ("ar_qk_norm_rope_args", tar.ArQkNormRopeArgs),
             ("ar_paged_attention_args", tar.ArPagedAttentionArgs)]
    body, want = "", []
    for c, py in pairs:
        body += f'printf("%zu\\n", sizeof({c}));\n'
        want.append(ctypes.sizeof(py))
        for name, *_ in py._fields_:
            body += f'printf("%zu\\n", offsetof({c}, {name}));\n'
            want.append(getattr(py, name).offset)
    src = tmp_path / "layout.c"
    src.write_text(f'#include <stdio.h>\n#include <stddef.h>\n#include "ar.h"\nint main(void) {{\n{body}return 0;\n}}\n')
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.run(["gcc", "-std=c11", "-I", include, str(src), "-o", str(tmp_path / "layout")], check=True)
    got = subprocess.run([str(tmp_path / "layout")], capture_output=True, text=True, check=True, timeout=60).stdout.split()
    assert [int(x) for x in got] == want


def test_packed_arguments_are_the_structures():
    """The bytes that the methods pass hold the fields where the structures do."""
    for args, pack in ((tar.ArPagedPlanArgs, tar._pack_plan), (tar.ArQkNormRopeArgs, tar._pack_rope),
                       (tar.ArPagedAttentionArgs, tar._pack_attention)):
        values, n = [], 0
        for _, kind in args._fields_:
            count = getattr(kind, "_length_", 1)
            values.append(tuple(range(n + 1, n + 1 + count)) if hasattr(kind, "_length_") else n + 1)
            n += count
        flat = [x for v in values for x in (v if isinstance(v, tuple) else (v,))]
        blob = pack(*flat)
        a = args.from_buffer_copy(blob + bytes(ctypes.sizeof(args) - len(blob)))
        for (name, kind), v in zip(args._fields_, values):
            got = getattr(a, name)
            assert (tuple(got) if isinstance(v, tuple) else got) == v, name
