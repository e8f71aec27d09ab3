"""What the attention block's methods hand to the C calls, without a GPU: host tensors (torch names their
device -1) and a recorder in the place of each C function."""
import ctypes

import pytest
import torch

import tensor_all_reduce_gb300 as tar


@pytest.fixture(scope="module", autouse=True)
def lib():
    from tensor_all_reduce_gb300 import _build
    _build.build()
    return tar.load_library()


class Host(tar.Context):
    """A context on no device, whose calls are recorded as argument structures."""

    ARGS = {"ar_paged_plan": tar.ArPagedPlanArgs, "ar_qk_norm_rope": tar.ArQkNormRopeArgs, "ar_paged_attention": tar.ArPagedAttentionArgs}

    def __init__(self):
        self.device, self.handle, self.calls = -1, None, []

    def _empty(self, shape, dtype, stream):
        return torch.empty(shape, dtype=dtype)

    def _call(self, name, packed, stream):
        args = self.ARGS[name]
        self.calls.append(args.from_buffer_copy(packed + bytes(ctypes.sizeof(args) - len(packed))))


def rotate(positions, sections, n=6, **kw):
    ctx = Host()
    q = torch.zeros(n, 2, 16, dtype=torch.bfloat16)
    ctx.qk_norm_rope(q, None, None, positions, torch.ones(8), sections=sections, **kw)
    return ctx.calls[-1]


@pytest.mark.parametrize("n", [1, 6])
@pytest.mark.parametrize("axes", [2, 3, 4])
@pytest.mark.parametrize("dealt", [False, True])
def test_positions_that_all_axes_share(n, axes, dealt):
    """An expanded row has one row of storage: no axis may be read behind it."""
    pos = torch.arange(n, dtype=torch.int32)
    a = rotate(pos.expand(axes, n), [8 - axes + 1] + [1] * (axes - 1), n, dealt=dealt)
    rows = a.axes if a.rot_dim else 0
    stride = a.position_stride or a.tokens
    assert a.positions == pos.data_ptr()
    assert (rows - 1) * stride + n <= pos.numel()


def test_sections_of_shared_positions_are_checked():
    pos = torch.arange(6, dtype=torch.int32).expand(3, 6)
    for sections in ([3, 3, 3], [9, -1, 0], [8, 8]):
        with pytest.raises((tar.ArError, ValueError)):
            rotate(pos, sections)


@pytest.mark.parametrize("n", [1, 6])
def test_rows_of_positions_apart(n):
    """Rows of a wider tensor keep their stride."""
    wide = torch.zeros(3, 50, dtype=torch.int32)
    a = rotate(wide[:, 7:7 + n], [3, 3, 2], n)
    assert (a.axes, a.position_stride, list(a.sections)[:3]) == (3, 50, [3, 3, 2])
    a = rotate(torch.zeros(3, n, dtype=torch.int32), [3, 3, 2], n)
    assert (a.axes, a.position_stride or a.tokens) == (3, n)
