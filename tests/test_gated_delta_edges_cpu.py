"""Edges of the gated delta rule's and the norm's calls that need no GPU: sizes near the end of an
int, and workspaces whose elements are not all there."""
import pytest
import torch

from linear_attention_rnn_finch_b200 import binding as bd
from linear_attention_rnn_finch_b200 import build

INT_MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    build.build()
    return bd.load()


@pytest.mark.parametrize("T", [INT_MAX, INT_MAX - 63])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_lengths_near_the_end_of_an_int(lib, T, dtype):
    """T + 63 would leave the ints: refused, and no bytes are asked for."""
    sizes = (1, T, 1, 1, 64)
    assert lib.gated_delta_prefill(*[None] * 5, 1.0, *[None] * 3, *sizes, bd._io(dtype), None, 0, None) == bd.WKV_ERR_UNSUPPORTED
    assert lib.gated_delta_backward(*[None] * 5, 1.0, *[None] * 9, *sizes, bd._io(dtype), None, 0, None) == bd.WKV_ERR_UNSUPPORTED
    assert bd.gated_delta_prefill_workspace_bytes(*sizes, dtype) == 0
    assert bd.gated_delta_backward_workspace_bytes(*sizes, dtype) == 0


def test_workspace_must_be_dense():
    """An expanded byte counts a thousand elements and has room for one."""
    one = torch.empty(1, dtype=torch.uint8)
    for bad in (one.expand(1024), torch.empty(64, 32, dtype=torch.uint8)[:, ::2]):
        with pytest.raises(ValueError):
            bd._workspace(bad, 256, "cpu")
    with pytest.raises(TypeError):
        bd._workspace(4096, 256, "cpu")
    ws, at, n = bd._workspace(torch.empty(100, dtype=torch.float32), 256, "cpu")
    assert at == ws.data_ptr() and n == 400
    assert bd._workspace(None, 0, "cpu") == (None, None, 0)


def test_sizes_that_ctypes_would_cut():
    bd._fits("channels", INT_MAX)
    with pytest.raises(ValueError):
        bd._fits("channels", 2 ** 32 + 64)
