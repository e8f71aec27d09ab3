"""Refusals, structure layouts and argument marshalling of the calls over a cache held in 8 bits, without a GPU: a call whose
arguments are right returns AR_ERR_NOT_INITIALIZED with ctx = NULL, a wrong one its own error, and nothing runs."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import serve8_ref as ref8
import tensor_all_reduce_gb300 as tar
from test_serve_host import AL, IA, NI, OV, UN, at
from test_serve_unprepared import unprepared  # noqa: F401  (a fixture)

D, T, HQ, HK, PG, NB = 128, 32, 12, 2, 16, 100


@pytest.fixture(scope="module", autouse=True)
def lib():
    from tensor_all_reduce_gb300 import _build
    _build.build()
    return tar.load_library()


def append(sections=(), ctx=None, **kw):
    row = 2 * HK * D
    d = dict(tokens=T, requests=4, kv_heads=HK, head_dim=D, dtype=tar.AR_DTYPE_BF16, k=at(0), v=at(0) + HK * D * 2, k_token_stride=row, k_head_stride=D,
             v_token_stride=row, v_head_stride=D, k_weight=at(1), eps=1e-6, gemma=0, rot_dim=D, pairs=0, axes=1, dealt=0, positions=at(2),
             position_stride=0, inv_freq=at(3), k_cache=at(4), v_cache=at(5), k_block_stride=PG * HK * D, k_page_stride=HK * D, k_cache_head_stride=D,
             v_block_stride=PG * HK * D, v_page_stride=HK * D, v_cache_head_stride=D, num_blocks=NB, page_size=PG, k_scale=at(6), v_scale=at(7),
             k_scale_block_stride=HK, k_scale_head_stride=1, v_scale_block_stride=HK, v_scale_head_stride=1, block_table=at(8), table_cols=10,
             table_stride=0, cu_q=at(9), seq_lens=at(10))
    d.update(kw)
    a = tar.ArPagedAppendFp8Args(**d)
    for i, n in enumerate(sections):
        a.sections[i] = n
    return tar.ar_paged_append_fp8(ctx, a, None, raise_on_error=False)


@pytest.mark.parametrize("want, kw", [
    (NI, {}), (NI, dict(tokens=0, k=None)), (NI, dict(requests=0)), (NI, dict(k_weight=None)), (NI, dict(rot_dim=0, positions=None, inv_freq=None)),
    (NI, dict(positions=None)), (NI, dict(axes=3, sections=(20, 22, 22))), (NI, dict(axes=2, sections=(64, 0), dealt=1)),
    (NI, dict(num_blocks=0, k_cache=None, v_cache=None, k_scale=None, v_scale=None)), (NI, dict(table_cols=0, block_table=None)),
    # one cache tensor [blocks, 2, page, heads, dim], scales [blocks, 2, heads], [heads, blocks]
    (NI, dict(k_block_stride=2 * PG * HK * D, v_block_stride=2 * PG * HK * D, v_cache=at(4) + PG * HK * D)),
    (NI, dict(k_scale_block_stride=2 * HK, v_scale_block_stride=2 * HK, v_scale=at(6) + 4 * HK)),
    (NI, dict(k_scale_block_stride=1, k_scale_head_stride=NB)), (NI, dict(k_cache=at(4) + 1, v_cache=at(5) + 3)),
    (NI, dict(num_blocks=1, k_scale_block_stride=0)), (NI, dict(kv_heads=1, k_scale_head_stride=0)),
    (IA, dict(tokens=-1)), (IA, dict(tokens=(1 << 30) + 1)), (IA, dict(requests=-1)), (IA, dict(requests=tar.AR_MAX_REQUESTS + 1)), (IA, dict(kv_heads=0)),
    (IA, dict(head_dim=0)), (IA, dict(head_dim=257)), (IA, dict(dtype=tar.AR_DTYPE_F32)), (IA, dict(eps=-1.0)), (IA, dict(eps=float("nan"))),
    (IA, dict(rot_dim=63)), (IA, dict(rot_dim=D + 2)), (IA, dict(axes=0)), (IA, dict(axes=5)), (IA, dict(axes=3, sections=(20, 22, 21))),
    (IA, dict(axes=2, sections=(65, -1))), (IA, dict(axes=2, sections=(32, 32), position_stride=T - 1)), (IA, dict(axes=2, sections=(32, 32), positions=None)),
    (IA, dict(k=None)), (IA, dict(v=None)), (IA, dict(inv_freq=None)), (IA, dict(k_cache=None)), (IA, dict(v_cache=None)), (IA, dict(k_scale=None)),
    (IA, dict(v_scale=None)), (IA, dict(block_table=None)), (IA, dict(cu_q=None)), (IA, dict(seq_lens=None)), (IA, dict(page_size=0)),
    (IA, dict(page_size=65537)), (IA, dict(num_blocks=-1)), (IA, dict(table_cols=-1)), (IA, dict(table_stride=9)), (IA, dict(k_head_stride=D - 1)),
    (IA, dict(v_token_stride=-1)), (IA, dict(k_cache_head_stride=1)), (IA, dict(k_scale_block_stride=0)), (IA, dict(v_scale_head_stride=0)),
    (IA, dict(k_scale_block_stride=1)), (IA, dict(v_scale_head_stride=-1)), (IA, dict(k_scale_block_stride=NB - 2, k_scale_head_stride=NB - 2)), (NI, dict(k_scale_block_stride=NB - 1, k_scale_head_stride=NB - 2)),
    (AL, dict(k=at(0) + 1)), (AL, dict(v=at(0) + 1)), (AL, dict(k_scale=at(6) + 2)), (AL, dict(v_scale=at(7) + 1)), (AL, dict(cu_q=at(9) + 2)),
    (AL, dict(positions=at(2) + 2)), (AL, dict(k_weight=at(1) + 1)), (AL, dict(block_table=at(8) + 1)),
    (OV, dict(v_cache=at(4))), (OV, dict(v_scale=at(6))), (OV, dict(k_cache=at(0))), (OV, dict(k_scale=at(4) + 64)), (OV, dict(v_scale=at(10))),
    (OV, dict(k_scale=at(8))), (OV, dict(v_cache=at(1))), (OV, dict(v_scale=at(6) + 4)), (OV, dict(k_cache=at(3))),
])
def test_append_refusals(want, kw):
    assert append(**kw) == want


def attention(ctx=None, **kw):
    d = dict(tokens=T, requests=4, q_heads=HQ, kv_heads=HK, head_dim=D, dtype=tar.AR_DTYPE_BF16, q=at(0), out=at(1), q_token_stride=HQ * D,
             q_head_stride=D, out_token_stride=HQ * D, out_head_stride=D, lse=at(2), k_cache=at(3), v_cache=at(4), k_block_stride=PG * HK * D,
             k_page_stride=HK * D, k_head_stride=D, v_block_stride=PG * HK * D, v_page_stride=HK * D, v_head_stride=D, num_blocks=NB, page_size=PG,
             block_table=at(5), table_cols=10, table_stride=0, cu_q=at(6), seq_lens=at(7), scale=0.1, causal=1, window=0, softcap=0.0, slopes=at(8),
             prefix_lens=at(9), workspace=at(10), workspace_bytes=1 << 30)
    s = dict(k_scale=at(30), v_scale=at(31), k_scale_block_stride=HK, k_scale_head_stride=1, v_scale_block_stride=HK, v_scale_head_stride=1)
    for n, v in kw.items():
        (s if n in s else d)[n] = v
    a = tar.ArPagedAttentionFp8Args(base=tar.ArPagedAttentionArgs(**d), **s)
    return tar.ar_paged_attention_fp8(ctx, a, None, raise_on_error=False)


@pytest.mark.parametrize("want, kw", [
    (NI, {}), (NI, dict(tokens=0)), (NI, dict(requests=0)), (NI, dict(lse=None, slopes=None, prefix_lens=None)), (NI, dict(window=1 << 30)),
    (NI, dict(num_blocks=0, k_cache=None, v_cache=None, k_scale=None, v_scale=None)), (NI, dict(softcap=30.0, causal=0)),
    (NI, dict(k_cache=at(3) + 1)), (NI, dict(k_scale_block_stride=0, k_scale_head_stride=0, v_scale=at(30))),
    (IA, dict(tokens=-1)), (IA, dict(requests=tar.AR_MAX_REQUESTS + 1)), (IA, dict(q_heads=13)), (IA, dict(head_dim=257)), (IA, dict(dtype=tar.AR_DTYPE_F32)),
    (IA, dict(scale=float("nan"))), (IA, dict(window=-1)), (IA, dict(page_size=0)), (IA, dict(table_stride=9)), (IA, dict(q=None)), (IA, dict(k_cache=None)),
    (IA, dict(k_scale=None)), (IA, dict(v_scale=None)), (IA, dict(k_scale_block_stride=-1)), (IA, dict(v_scale_head_stride=-2)), (IA, dict(workspace=None)),
    (UN, dict(tokens=1 << 30)),
    (AL, dict(q=at(0) + 1)), (AL, dict(k_scale=at(30) + 2)), (AL, dict(v_scale=at(31) + 1)), (AL, dict(workspace=at(10) + 8)),
    (OV, dict(out=at(0))), (OV, dict(out=at(3) + 64)), (OV, dict(out=at(30))), (OV, dict(lse=at(31) + 16)), (OV, dict(workspace=at(30))),
])
def test_attention_refusals(want, kw):
    assert attention(**kw) == want


@pytest.mark.parametrize("call", [append, attention])
def test_an_unprepared_context_says_so(unprepared, call):  # noqa: F811
    ctx = ctypes.addressof(unprepared)
    assert call(ctx=ctx) == tar.AR_ERR_CUDA and "attention block" in tar.ar_last_error(ctx)
    assert call(ctx=ctx, tokens=0) == tar.AR_OK


def test_null_arguments():
    lib = tar.load_library()
    assert lib.ar_paged_append_fp8(None, None, None) == IA and lib.ar_paged_attention_fp8(None, None, None) == IA


def test_argument_blocks_match_the_header(tmp_path):
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    body, want = "", []
    for c, py in (("ar_paged_append_fp8_args", tar.ArPagedAppendFp8Args), ("ar_paged_attention_fp8_args", tar.ArPagedAttentionFp8Args)):
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


class Host(tar.Context):
    """A context on no device, whose calls are recorded as argument structures."""

    def __init__(self):
        self.device, self.handle, self.calls = -1, None, []

    def _empty(self, shape, dtype, stream):
        return torch.empty(shape, dtype=dtype)

    def _call(self, name, packed, stream):
        args = {"ar_paged_append_fp8": tar.ArPagedAppendFp8Args, "ar_paged_attention_fp8": tar.ArPagedAttentionFp8Args}[name]
        assert len(packed) <= ctypes.sizeof(args)
        self.calls.append(args.from_buffer_copy(packed + bytes(ctypes.sizeof(args) - len(packed))))


def test_what_the_methods_hand_over():
    ctx = Host()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    kv = torch.zeros(6, 4, 16, dtype=torch.float16)
    cache = torch.zeros(5, 2, 8, 2, 16, dtype=torch.uint8).view(torch.float8_e4m3fn)
    scale = torch.zeros(2, 3, 5)
    table, cu, lens, pos, freq = torch.zeros(2, 9, dtype=torch.int32)[:, :7], i32(0, 2, 6), i32(7, 6), torch.zeros(2, 50, dtype=torch.int32)[:, 3:9], torch.ones(8)
    ctx.paged_append_fp8(kv[:, :2], kv[:, 2:], cache[:, 0], cache[:, 1].view(torch.uint8), scale[:, 0].t(), scale[:, 1].t(), table, cu, lens, positions=pos,
                         inv_freq=freq, eps=0.5, gemma=True, pairs=True, sections=[5, 3], dealt=True)
    a = ctx.calls[-1]
    assert (a.tokens, a.requests, a.kv_heads, a.head_dim, a.dtype) == (6, 2, 2, 16, tar.AR_DTYPE_F16)
    assert (a.k, a.v, a.k_token_stride, a.v_head_stride) == (kv.data_ptr(), kv.data_ptr() + 64, 64, 16)
    assert (a.k_weight, a.eps, a.gemma, a.rot_dim, a.pairs, a.axes, list(a.sections), a.dealt) == (None, 0.5, 1, 16, 1, 2, [5, 3, 0, 0], 1)
    assert (a.positions, a.position_stride, a.inv_freq) == (pos.data_ptr(), 50, freq.data_ptr())
    assert (a.k_cache, a.v_cache, a.k_block_stride, a.k_page_stride, a.v_cache_head_stride) == (cache.data_ptr(), cache.data_ptr() + 256, 512, 32, 16)
    assert (a.num_blocks, a.page_size, a.k_scale, a.v_scale) == (5, 8, scale.data_ptr(), scale.data_ptr() + 20)
    assert (a.k_scale_block_stride, a.k_scale_head_stride, a.v_scale_block_stride, a.v_scale_head_stride) == (1, 15, 1, 15)
    assert (a.block_table, a.table_cols, a.table_stride, a.cu_q, a.seq_lens) == (table.data_ptr(), 7, 9, cu.data_ptr(), lens.data_ptr())
    ctx.paged_append_fp8(kv[:, :2], kv[:, 2:], cache[:, 0], cache[:, 1], scale[:, 0].t(), scale[:, 1].t(), table, cu, lens, inv_freq=freq)
    a = ctx.calls[-1]
    assert (a.positions, a.axes, a.rot_dim, a.gemma, a.dealt) == (None, 1, 16, 0, 0)
    q, work = torch.zeros(6, 4, 16, dtype=torch.bfloat16), torch.empty(64, dtype=torch.uint8)
    ctx.paged_attention_fp8(q, cache[:, 0], cache[:, 1], scale[:, 0].t(), scale[:, 1].t(), table, cu, lens, window=3, softcap=2.0, workspace=work)
    a = ctx.calls[-1]
    b = a.base
    assert (b.tokens, b.requests, b.q_heads, b.kv_heads, b.head_dim, b.window, b.softcap, b.scale) == (6, 2, 4, 2, 16, 3, 2.0, 0.25)
    assert (b.k_cache, b.v_block_stride, b.num_blocks, b.workspace, b.workspace_bytes) == (cache.data_ptr(), 512, 5, work.data_ptr(), 64)
    assert (a.k_scale, a.v_scale, a.k_scale_head_stride, a.v_scale_block_stride) == (scale.data_ptr(), scale.data_ptr() + 20, 15, 1)


def test_rounding_of_the_reference():
    """serve8_ref's rounding to E4M3 and scales: every code, midpoints with ties to even, and 448's borders."""
    codes = torch.arange(256, dtype=torch.uint8).view(ref8.E4M3).double()
    codes = codes[~codes.isnan()]
    assert torch.equal(ref8.round_e4m3(codes), codes)
    x = torch.cat([torch.linspace(-470, 470, 20001, dtype=torch.float64), torch.linspace(-0.04, 0.04, 20001, dtype=torch.float64)])
    pos = codes[codes >= 0].sort().values.unique()
    x = torch.cat([x, (pos[1:] + pos[:-1]) / 2])
    want = x.float().clamp(-448, 448).to(ref8.E4M3).double()
    assert torch.equal(ref8.round_e4m3(x), want)
    for top, s in ((448.0, 1.0), (448.0000001, 2.0), (447.9, 1.0), (224.0, 0.5), (1e-30, 2.0 ** -32), (0.0, 2.0 ** -32), (1e30, 2.0 ** 32), (3.5, 2.0 ** -7)):
        assert ref8.fresh(top) == s
