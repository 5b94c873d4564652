"""The gated delta rule and group norm with an activation on a stream given by `stream=`: a
workspace that the call allocates itself stays its own until the stream has come to it, whatever
the current stream allocates and writes meanwhile."""
import pytest
import torch

import linear_attention_rnn_finch_b200 as gw
from tests.test_gated_delta_gpu import BF16, DEV, SCALE, args, problem

pytestmark = pytest.mark.gpu
F32 = torch.float32


def delta(B, T, H, HK, dtype, backward):
    p = problem(900 + T, B, T, H, HK, dtype)
    a = args(p)
    if not backward:
        return lambda **kw: gw.gated_delta_prefill(*a, scale=SCALE, **kw)
    dy = torch.randn_like(a[2])
    return lambda **kw: gw.gated_delta_backward(*a[:6], dy, scale=SCALE, **kw)


def norm(N, L, C, dtype, backward):
    g = torch.Generator(device=DEV).manual_seed(N * L)
    x, dy = (torch.randn(N, L, C, generator=g, device=DEV).to(dtype) for _ in range(2))
    gamma, beta = (torch.randn(C, generator=g, device=DEV) for _ in range(2))
    if not backward:
        return lambda **kw: (gw.group_norm_act(x, gamma, beta, groups=4, **kw),)
    return lambda **kw: gw.group_norm_act_backward(x, gamma, beta, 1e-5, dy, groups=4, **kw)[:3]


@pytest.mark.parametrize("make,sizes", [
    (delta, (1, 2048, 1, 1, BF16, False)), (delta, (1, 333, 4, 2, F32, True)),
    (delta, (1, 200, 4, 2, BF16, True)), (norm, (2, 1021, 64, BF16, False)),
    (norm, (2, 1021, 64, F32, True)), (norm, (300, 1, 64, BF16, True))])
def test_workspace_of_a_waiting_stream(make, sizes):
    call = make(*sizes)
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)   # some 10 ms, in which the host runs on
    got = call(stream=side)
    # what the current stream's pool has to give, overwritten at once
    mine = [torch.full((1 << n,), float("nan"), device=DEV) for n in (8, 12, 16, 18, 20) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.isnan(m).all() for m in mine)
    for a, b in zip(got, want):
        assert (a is None and b is None) or torch.equal(a, b)


def test_stream_of_the_call_is_the_current_one_again():
    side, now = torch.cuda.Stream(), torch.cuda.current_stream()
    norm(2, 40, 64, F32, False)(stream=side)
    assert torch.cuda.current_stream() == now
    torch.cuda.synchronize()
