"""Edges of the gated delta rule's and the norm's calls on the GPU: key heads without value heads,
sizes beyond 32 bits, padding, and waits that expire on a full device."""
import ctypes

import pytest
import torch

import linear_attention_rnn_finch_b200 as gw
from linear_attention_rnn_finch_b200 import binding as bd
from tests import gated_delta_ref as ref
from tests.gated_delta_ref import OWN, c64, close
from tests.test_gated_delta_gpu import BF16, DEV, F32, SCALE, args, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_key_heads_without_value_heads(dtype):
    """dq and dk are each key head's sum over no value heads: zeros, whatever lay there before."""
    L = bd.load()
    B, T, HK = 2, 70, 3
    q, k = (torch.randn(B, T, HK, 64, device=DEV).to(dtype) for _ in range(2))
    dq, dk = (torch.full_like(q, float("nan")) for _ in range(2))
    at = lambda t: ctypes.c_void_p(t.data_ptr())

    def call(a, b):
        st = L.gated_delta_backward(at(q), at(k), None, None, None, 1.0, None, None, None, a, b, None, None, None,
                                    None, B, T, 0, HK, 64, bd._io(dtype), None, 0, None)
        torch.cuda.synchronize()
        return st

    assert call(None, at(dk)) == bd.WKV_ERR_INVALID_ARG and call(at(q), at(dk)) == bd.WKV_ERR_INVALID_ARG
    assert call(at(dq), at(dq)) == bd.WKV_ERR_INVALID_ARG
    assert bool(torch.isnan(dq).all()) and bool(torch.isnan(dk).all())
    assert call(at(dq), at(dk)) == bd.WKV_OK
    assert bool((dq == 0).all()) and bool((dk == 0).all())
    v, om = torch.empty(B, T, 0, 64, device=DEV, dtype=dtype), torch.empty(B, T, 0, device=DEV, dtype=dtype)
    held = [torch.full_like(q, float("nan")) for _ in range(4)]
    torch.cuda.synchronize()
    del held
    out = gw.gated_delta_backward(q, k, v, om, om.clone(), None, v.clone())
    assert bool((out[0] == 0).all()) and bool((out[1] == 0).all())
    y, s = gw.gated_delta_prefill(q, k, v, om, om.clone())
    assert y.shape == (B, T, 0, 64) and s.shape == (B, 0, 64, 64)


def test_channels_beyond_32_bits_are_refused():
    """2^32 + 64 channels are 64 in a C int."""
    C = 2 ** 32 + 64
    x = torch.empty(1, C, device=DEV, dtype=BF16)
    p = torch.empty(C, device=DEV)
    with pytest.raises(ValueError):
        gw.group_norm_act(x, p, p.clone(), groups=1)
    with pytest.raises(ValueError):
        gw.group_norm_act_backward(x, p, p.clone(), 1e-5, x.clone(), groups=1)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("side", ["left", "right"])
def test_padding_on_either_side(side, dtype):
    """Tokens with beta = 0 and omega = -inf, q, k and v zeros or another token's: the others' outputs
    and the state are those of the recurrence without them."""
    B, T, n = 2, 150, 37
    p = problem(700, B, T, 4, 2, dtype)
    for fill in ("zeros", "others"):
        pad = {}
        for name in ("q", "k", "v", "omega", "beta"):
            x = p[name][:, :n].clone()
            if name == "omega":
                x.fill_(-float("inf"))
            elif name == "beta" or fill == "zeros":
                x.zero_()
            pad[name] = torch.cat([x, p[name]] if side == "left" else [p[name], x], 1).contiguous()
        pad["s0"] = p["s0"]
        y0, s0 = ref.prefill(*[c64(a) for a in args(p)], scale=SCALE)
        y1, s1 = gw.gated_delta_prefill(*args(pad), scale=SCALE)
        own = y1[:, n:] if side == "left" else y1[:, :T]
        close(own.contiguous(), y0, OWN[dtype], "y")
        close(s1, s0, OWN[dtype], "state")


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
