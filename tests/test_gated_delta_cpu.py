"""The gated delta rule's and the norm's entry points without a GPU: exported symbols, workspace
queries, size checks (made before any device call) and the binding's refusals; and the 64-bit
reference forms the GPU tests use, against their definitions."""
import ctypes
import pathlib
import re

import pytest
import torch

import linear_attention_rnn_finch_b200 as gw
from linear_attention_rnn_finch_b200 import binding as bd
from linear_attention_rnn_finch_b200 import build
from tests import gated_delta_ref as ref

ROOT = pathlib.Path(__file__).resolve().parents[1]


def declared():
    text = re.sub(r"/\*.*?\*/", "", (ROOT / "include" / "goldwkv.h").read_text(), flags=re.S)
    return sorted(set(re.findall(r"\b((?:gated_delta|group_norm_act)\w*)\s*\(", text)))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return bd.load()


def test_declared_and_exported(lib):
    names = declared()
    assert {"gated_delta_prefill", "gated_delta_decode_step", "gated_delta_backward", "group_norm_act",
            "group_norm_act_backward"} <= set(names)
    raw = ctypes.CDLL(str(bd.LIB_PATH))
    for n in names:
        assert hasattr(raw, n), n


def test_public_names():
    for n in ("gated_delta_prefill", "gated_delta_decode_step", "gated_delta_backward", "group_norm_act",
              "group_norm_act_backward", "gated_delta_prefill_workspace_bytes",
              "gated_delta_backward_workspace_bytes", "group_norm_act_workspace_bytes"):
        assert n in gw.__all__ and callable(getattr(gw, n))


def test_workspace_queries(lib):
    assert bd.gated_delta_backward_workspace_bytes(1, 64, 2, 2, 64, torch.float32) > 0
    assert bd.gated_delta_prefill_workspace_bytes(1, 64, 2, 2, 64, torch.float32) == 0   # the recurrence
    for sizes in ((0, 64, 2, 2, 64), (1, 0, 2, 2, 64), (1, 64, 0, 0, 64), (1, 64, 4, 3, 64), (1, 64, 2, 2, 32),
                  (-1, 64, 2, 2, 64)):
        assert bd.gated_delta_backward_workspace_bytes(*sizes, torch.bfloat16) == 0
        assert bd.gated_delta_prefill_workspace_bytes(*sizes, torch.bfloat16) == 0
    assert bd.group_norm_act_workspace_bytes(100, 1, 64, 2, torch.bfloat16) == 0
    assert bd.group_norm_act_workspace_bytes(100, 1, 64, 2, torch.bfloat16, backward=True) > 0
    assert bd.group_norm_act_workspace_bytes(3, 10, 64, 2, torch.bfloat16) > 0
    assert bd.group_norm_act_workspace_bytes(3, 10, 64, 5, torch.bfloat16) == 0
    assert bd.group_norm_act_workspace_bytes(0, 10, 64, 2, torch.bfloat16) == 0


@pytest.mark.parametrize("sizes,io,scale,want", [
    ((2, 20, 4, 2, 32), 1, 1.0, bd.WKV_ERR_UNSUPPORTED),
    ((2, 20, 4, 3, 64), 1, 1.0, bd.WKV_ERR_INVALID_ARG),
    ((2, 20, 4, 0, 64), 1, 1.0, bd.WKV_ERR_INVALID_ARG),
    ((2, -1, 4, 2, 64), 1, 1.0, bd.WKV_ERR_INVALID_ARG),
    ((2, 20, 4, 2, 64), 9, 1.0, bd.WKV_ERR_INVALID_ARG),
    ((2, 20, 4, 2, 64), 1, float("nan"), bd.WKV_ERR_INVALID_ARG),
    ((1000, 2_000_000_000, 4, 2, 64), 1, 1.0, bd.WKV_ERR_UNSUPPORTED),
    ((0, 20, 4, 2, 64), 1, 1.0, bd.WKV_OK),
])
def test_size_checks(lib, sizes, io, scale, want):
    B, T, H, HK, D = sizes
    assert lib.gated_delta_prefill(*[None] * 5, scale, *[None] * 3, *sizes, io, None, 0, None) == want
    assert lib.gated_delta_backward(*[None] * 5, scale, *[None] * 9, *sizes, io, None, 0, None) == want
    if T == 20:
        assert lib.gated_delta_decode_step(*[None] * 5, scale, None, None, B, H, HK, D, io, None) == want


@pytest.mark.parametrize("sizes,eps,act,io,want", [
    ((3, 10, 64, 5), 1e-5, 1, 1, bd.WKV_ERR_INVALID_ARG),
    ((3, 10, 64, 0), 1e-5, 1, 1, bd.WKV_ERR_INVALID_ARG),
    ((3, 10, 0, 1), 1e-5, 1, 1, bd.WKV_ERR_INVALID_ARG),
    ((-3, 10, 64, 2), 1e-5, 1, 1, bd.WKV_ERR_INVALID_ARG),
    ((3, 10, 64, 2), 0.0, 1, 1, bd.WKV_ERR_INVALID_ARG),
    ((3, 10, 64, 2), float("nan"), 1, 1, bd.WKV_ERR_INVALID_ARG),
    ((3, 10, 64, 2), 1e-5, 5, 1, bd.WKV_ERR_INVALID_ARG),
    ((3, 10, 64, 2), 1e-5, 1, 5, bd.WKV_ERR_INVALID_ARG),
    ((1 << 40, 10, 64, 2), 1e-5, 1, 1, bd.WKV_ERR_UNSUPPORTED),
    ((0, 10, 64, 2), 1e-5, 1, 1, bd.WKV_OK),
])
def test_norm_size_checks(lib, sizes, eps, act, io, want):
    assert lib.group_norm_act(None, None, None, eps, act, None, None, *sizes, io, None, 0, None) == want


def test_binding_rejects_cpu_tensors():
    z = lambda *s: torch.zeros(s)
    with pytest.raises(ValueError):
        gw.gated_delta_prefill(z(1, 2, 1, 64), z(1, 2, 1, 64), z(1, 2, 1, 64), z(1, 2, 1), z(1, 2, 1))
    with pytest.raises(ValueError):
        gw.gated_delta_decode_step(z(1, 1, 64), z(1, 1, 64), z(1, 1, 64), z(1, 1), z(1, 1), z(1, 1, 64, 64))
    with pytest.raises(ValueError):
        gw.group_norm_act(z(4, 64), z(64), z(64), groups=2)
    with pytest.raises(TypeError):
        gw.gated_delta_prefill(None, z(1, 2, 1, 64), z(1, 2, 1, 64), z(1, 2, 1), z(1, 2, 1))


# ------------------------------------------------------------------ the reference forms

def _small(T=6, D=64):
    g = torch.Generator().manual_seed(0)
    rn = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    k = rn(1, T, 1, D)
    return rn(1, T, 1, D), k / k.norm(dim=-1, keepdim=True), rn(1, T, 2, D), rn(1, T, 2), torch.rand(1, T, 2, dtype=torch.float64)


def test_reference_no_decay_full_strength_recalls():
    """omega = -inf, beta = 1, orthonormal keys: reading with a key returns its value."""
    q, k, v, om, be = _small()
    k = torch.linalg.qr(k[0, :, 0].T)[0].T[None, :, None]
    om, be = torch.full_like(om, -float("inf")), torch.ones_like(be)
    _, S = ref.prefill(k, k, v, om, be)
    for t in range(6):
        assert torch.allclose(torch.einsum("hij,i->hj", S[0], k[0, t, 0]), v[0, t])


def test_reference_overwrites_at_strength_one():
    """A unit key written twice at beta = 1 holds the second value only."""
    q, k, v, om, be = _small(2)
    k = k[:, :1].expand(1, 2, 1, 64)
    _, S = ref.prefill(k, k, v, torch.full_like(om, -2.0), torch.ones_like(be))
    assert torch.allclose(torch.einsum("hij,i->hj", S[0], k[0, 0, 0]), v[0, 1])


def test_reference_matrix_form():
    """S_t = w (I - b k k^T) S_{t-1} + b k v^T."""
    q, k, v, om, be = _small()
    _, S = ref.prefill(q, k, v, om, be)
    M = torch.zeros(64, 64, dtype=torch.float64)
    for t in range(6):
        kk, b, w = k[0, t, 0][:, None], be[0, t, 1], torch.exp(-torch.exp(om[0, t, 1]))
        M = w * (torch.eye(64, dtype=torch.float64) - b * kk @ kk.T) @ M + b * kk @ v[0, t, 1][None]
    assert torch.allclose(S[0, 1], M)


def test_reference_group_norm_moments():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 7, 12, generator=g, dtype=torch.float64) + 5
    y = ref.group_norm(x, torch.ones(12, dtype=torch.float64), torch.zeros(12, dtype=torch.float64), 1e-14, 3, "none")
    h = y.view(3, 7, 3, 4)
    assert h.mean((1, 3)).abs().max() < 1e-12
    assert (h.pow(2).mean((1, 3)) - 1).abs().max() < 1e-12
