"""Calls over an 8-bit cache that have nothing to do: a step without tokens or requests, whose empty arrays have no address, is no
error whatever else the call asks for.  Without a GPU: AR_ERR_NOT_INITIALIZED with ctx = NULL is what a call without faults gives."""
import pytest

from test_fp8_host import append, attention, lib  # noqa: F401  (a fixture)
from test_serve_host import IA, NI

NOTHING = dict(k=None, v=None, positions=None)


@pytest.mark.parametrize("axes, sections", [(1, ()), (2, (32, 32)), (3, (20, 22, 22)), (4, (16, 16, 16, 16))])
def test_append(axes, sections):
    for kw in (dict(tokens=0, **NOTHING), dict(tokens=0, requests=0, cu_q=None, seq_lens=None, block_table=None, **NOTHING),
               dict(requests=0, seq_lens=None, block_table=None)):
        assert append(axes=axes, sections=sections, **kw) == NI
    assert append(axes=axes, sections=sections, positions=None) == (NI if axes == 1 else IA)  # each token's place is one axis


def test_attention():
    for kw in (dict(tokens=0, q=None, out=None), dict(requests=0, seq_lens=None, block_table=None)):
        assert attention(**kw) == NI
