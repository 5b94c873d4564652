"""Edges of the gated delta rule's and the norm's calls on the GPU."""
import pytest
import torch

import linear_attention_rnn_finch_b200 as gw
from tests.test_gated_delta_gpu import BF16, SCALE, args, problem

pytestmark = pytest.mark.gpu


def test_expired_waits_on_a_full_device():
    """With no cycles to wait in, four times: blocks are NaN or what they are, with two of them on
    an SM whose neighbours leave early, and the calls after it are whole."""
    p = problem(710, 4, 1000, 16, 8, BF16)
    dy = torch.randn_like(p["v"])
    want = gw.gated_delta_backward(*args(p), dy, scale=SCALE)
    with pytest.MonkeyPatch.context() as m:
        m.setenv("GOLDWKV_FAULT", "timeout0")
        late = [gw.gated_delta_backward(*args(p), dy, scale=SCALE) for _ in range(4)]
        torch.cuda.synchronize()
    whole = gw.gated_delta_backward(*args(p), dy, scale=SCALE)
    for got in late:
        assert bool(torch.isnan(got[0]).any())
        for i in (0, 1, 3, 4):
            assert torch.equal(torch.where(torch.isnan(got[i]), want[i], got[i]), want[i])
        assert torch.equal(got[2], want[2]) and torch.equal(got[5], want[5])
    for a, b in zip(whole, want):
        assert torch.equal(a, b)
