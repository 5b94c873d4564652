"""Edges of the gated delta rule's and the norm's calls that need no GPU."""
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
