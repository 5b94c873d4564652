"""Long sequences of few heads, which the bf16 calls cut into segments: against the plain 64-bit
recurrence, with the state in place, with decays of none and of everything at the borders, and
replayed."""
import pytest
import torch

import linear_attention_rnn_finch_b200 as gw
from linear_attention_rnn_finch_b200 import binding as bd
from tests import gated_delta_ref as ref
from tests.gated_delta_ref import OWN, c64, close
from tests.test_gated_delta_gpu import BF16, DEV, SCALE, args, check_backward, check_prefill, problem

pytestmark = pytest.mark.gpu

# (B, H, HK, T): one head, an odd end, several key heads, rows of a batch
SIZES = [(1, 1, 1, 1024), (1, 2, 1, 1801), (2, 3, 3, 1500), (1, 8, 2, 2051)]


def cut(B, T, H, HK):
    """A prefill that needs a workspace is one that is cut."""
    return bd.gated_delta_prefill_workspace_bytes(B, T, H, HK, 64, BF16) > 0


@pytest.mark.parametrize("B,H,HK,T", SIZES)
@pytest.mark.parametrize("decay,state", [("slow", True), ("usual", False)])
def test_prefill(B, H, HK, T, decay, state):
    assert cut(B, T, H, HK)
    check_prefill(problem(300 + T, B, T, H, HK, BF16, decay, state), BF16)


@pytest.mark.parametrize("decay", ["mixed", "ends"])
def test_prefill_decays(decay):
    check_prefill(problem(310, 1, 1500, 2, 2, BF16, decay), BF16)


def test_the_state_may_be_updated_in_place():
    B, H, HK, T = SIZES[1]
    p = problem(320, B, T, H, HK, BF16, "slow")
    yo, so = ref.prefill(*[c64(a) for a in args(p)], scale=SCALE)
    s = p["s0"].clone()
    y, out = gw.gated_delta_prefill(*args(p)[:5], s, scale=SCALE, state_out=s)
    assert out is s
    close(y, yo, OWN[BF16], "y")
    close(s, so, OWN[BF16], "state")


def test_in_pieces_of_any_length():
    """A cut call after a whole one and before another hands the same states on."""
    B, H, HK, T = 1, 2, 1, 2000
    p = problem(330, B, T, H, HK, BF16, "slow")
    yo, so = ref.prefill(*[c64(a) for a in args(p)], scale=SCALE)
    s, ys = p["s0"].clone(), []
    for a, b in ((0, 100), (100, 1700), (1700, 2000)):
        y, s = gw.gated_delta_prefill(*[p[n][:, a:b].contiguous() for n in ("q", "k", "v", "omega", "beta")], s, scale=SCALE)
        ys.append(y)
    close(torch.cat(ys, 1), yo, OWN[BF16], "y")
    close(s, so, 2 * OWN[BF16], "state")   # three calls' states, each off by its own share


@pytest.mark.parametrize("B,H,HK,T", SIZES)
@pytest.mark.parametrize("decay,state,ds", [("slow", True, True), ("usual", False, True), ("slow", True, False)])
def test_backward(B, H, HK, T, decay, state, ds):
    check_backward(problem(340 + T, B, T, H, HK, BF16, decay, state), BF16, ds=ds)


@pytest.mark.parametrize("decay", ["mixed", "ends"])
def test_backward_decays(decay):
    check_backward(problem(350, 1, 1500, 2, 2, BF16, decay), BF16)


def test_same_bits_replayed():
    B, H, HK, T = SIZES[3]
    p = problem(360, B, T, H, HK, BF16)
    dy = torch.randn_like(p["v"])

    def calls():
        y, s = gw.gated_delta_prefill(*args(p), scale=SCALE)
        return [y, s, *gw.gated_delta_backward(*args(p), dy, s, scale=SCALE)]

    want = [x.clone() for x in calls()]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = calls()
    for _ in range(2):
        for x in outs:
            x.zero_()
        g.replay()
        for x, y in zip(want, outs):
            assert torch.equal(x, y)


def test_a_wait_that_expires_leaves_nan(monkeypatch):
    """With no cycles to wait in, the blocks whose products are not done at once are NaN, the
    others what they are; the call after it is whole again."""
    p = problem(370, 2, 130, 4, 2, BF16)
    dy = torch.randn_like(p["v"])
    want = gw.gated_delta_backward(*args(p), dy, scale=SCALE)
    monkeypatch.setenv("GOLDWKV_FAULT", "timeout0")
    got = gw.gated_delta_backward(*args(p), dy, scale=SCALE)
    torch.cuda.synchronize()
    monkeypatch.delenv("GOLDWKV_FAULT")
    assert bool(torch.isnan(got[0]).any())
    for i in (0, 1, 3, 4):
        nan = torch.isnan(got[i])
        assert torch.equal(torch.where(nan, want[i], got[i]), want[i])
        # whole blocks of 64 tokens: 0-63, 64-127, 128-129
        for a, b in ((0, 64), (64, 128), (128, 130)):
            per_head = nan[:, a:b].flatten(3).all(3).all(1) if nan.dim() == 4 else nan[:, a:b].all(1)
            some = nan[:, a:b].flatten(3).any(3).any(1) if nan.dim() == 4 else nan[:, a:b].any(1)
            assert torch.equal(per_head, some)
    assert torch.equal(got[2], want[2]) and torch.equal(got[5], want[5])   # dv, dstate: no such wait
    for x, y in zip(gw.gated_delta_backward(*args(p), dy, scale=SCALE), want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("B,H,HK,T", [(37, 4, 2, 35), (149, 1, 1, 17)])
def test_prefill_of_many_heads(B, H, HK, T, dtype):
    """From 148 heads on, where fp32 takes all 64 value columns in one block of threads."""
    check_prefill(problem(380, B, T, H, HK, dtype), dtype)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_backward_of_many_heads(dtype):
    """76 heads: fp32 takes all 64 value columns of a head in one block of threads, as from 10 on."""
    check_backward(problem(390, 19, 70, 4, 2, dtype), dtype)
