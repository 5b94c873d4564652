"""How exactly the calls keep what they hold and return in fp32, the state and the initial state's
gradient, over long sequences that forget slowly or not at all, whole and cut into segments,
against the 64-bit recurrence.

Tolerances, of the tensor's norm.  For |k| = 1, 0 <= beta <= 2 and w <= 1 a token's map of the
state does not expand, so errors made on the way are at most carried along.  16 tokens round the
state about five times (the products with keys, with the triangular inverse and of the update,
two sums), each by at most 2^-24, with signs that are independent: n times 16 tokens that are
remembered leave sqrt(n) 5 x 2^-24.
  beta = 0.9 or the sigmoid of a normal number: a token leaves 0.01 (on average 0.3) of the energy
    along its key, one of 64 directions, so that 64 / 0.99 to 64 / 0.7 = 91 tokens are remembered,
    n < 6, 7.3e-7; 1e-6 also covers what the values of the last tokens add.
  Nothing forgotten (beta = 2, no decay, a reflection): n = T / 16, 4.8e-6 at 4096 tokens.  Tensor
    cores may cut their sums off instead of rounding them, up to 2^-23 and on average 2^-24 of a
    value, always towards zero, and the update of the state is what three products in a row leave.
    16 tokens' update U has the norm of S (4 |k^T S|^2 = 4 / 64 of |S|^2 a token) and leaves |S| as it
    is, 2 <S, U> = -|U|^2; one that is cut by c of itself leaves |S + (1 - c) U|^2 = |S|^2 - c |U|^2, c / 2 of
    |S| less, and c = 3 x 2^-24.  The same way every time, n of them leave n 3 x 2^-25, 2.3e-5 at
    4096 tokens.
"""
import pytest
import torch

import linear_attention_rnn_finch_b200 as gw
from linear_attention_rnn_finch_b200 import binding as bd
from tests import gated_delta_ref as ref
from tests.test_gated_delta_gpu import BF16, DEV, SCALE, args, problem

pytestmark = pytest.mark.gpu


def long_problem(kind, B, T, H, HK):
    p = problem(500 + T, B, T, H, HK, BF16, "usual" if kind == "usual" else "slow")
    if kind in ("full", "reflect"):
        p["omega"].fill_(-float("inf"))
        p["beta"].fill_(0.9 if kind == "full" else 2.0)
    return p


def tolerance(kind, T, cut=True):
    """cut: the sums are tensor cores'."""
    n = T / 16
    return n ** 0.5 * 5 * 2.0 ** -24 + (n * 3 * 2.0 ** -25 if cut else 0) if kind == "reflect" else 1e-6


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


# (B, H, HK, T, cut into segments)
SIZES = [(1, 2, 1, 4096, True), (1, 160, 2, 1024, False)]
KINDS = ["usual", "slow", "full", "reflect"]


@pytest.mark.parametrize("B,H,HK,T,cut", SIZES)
@pytest.mark.parametrize("kind", KINDS)
def test_final_state(kind, B, H, HK, T, cut):
    assert (bd.gated_delta_prefill_workspace_bytes(B, T, H, HK, 64, BF16) > 0) == cut
    p = long_problem(kind, B, T, H, HK)
    _, s = gw.gated_delta_prefill(*args(p), scale=SCALE)
    _, want = ref.prefill(*[a.double() for a in args(p)], scale=SCALE)
    assert off(s, want) <= tolerance(kind, T)


@pytest.mark.parametrize("B,H,HK,T", [(1, 2, 1, 2048), (1, 160, 2, 256)])
@pytest.mark.parametrize("kind", KINDS)
def test_initial_state_gradient(kind, B, H, HK, T):
    """dstate_in runs through the same maps backward: the gradient G of the state meets K, T and
    the update as the state does."""
    p = long_problem(kind, B, T, H, HK)
    g = torch.Generator(device=DEV).manual_seed(2)
    dy = torch.randn(p["v"].shape, generator=g, device=DEV).to(BF16)
    dS = 0.3 * torch.randn((B, H, 64, 64), generator=g, device=DEV)
    got = gw.gated_delta_backward(*args(p), dy, dS, scale=SCALE)[5]
    # the adjoint of the recurrence, token by token
    q, k = (p[n].double().repeat_interleave(H // HK, 2) for n in ("q", "k"))
    w, beta, d = torch.exp(-torch.exp(p["omega"].double())), p["beta"].double(), dy.double()
    G = dS.double()
    for t in range(T - 1, -1, -1):
        G = G + SCALE * torch.einsum("bhi,bhj->bhij", q[:, t], d[:, t])
        de = beta[:, t, :, None] * torch.einsum("bhij,bhi->bhj", G, k[:, t])
        G = (G - torch.einsum("bhi,bhj->bhij", k[:, t], de)) * w[:, t, :, None, None]
    assert off(got, G) <= tolerance(kind, T)


@pytest.mark.parametrize("B,H,HK,T", [(1, 2, 1, 4096), (1, 160, 2, 1024)])
@pytest.mark.parametrize("kind", KINDS)
def test_final_state_token_by_token(kind, B, H, HK, T):
    """The fp32 prefill: a token's decay and update round each entry twice, 16 tokens 32 times by 2^-25
    on average, sqrt(32) 2^-25 = 2.9 x 2^-24 in all: within the tolerance of the others."""
    p = {n: x.float() for n, x in long_problem(kind, B, T, H, HK).items()}
    _, s = gw.gated_delta_prefill(*args(p), scale=SCALE)
    _, want = ref.prefill(*[a.double() for a in args(p)], scale=SCALE)
    assert off(s, want) <= tolerance(kind, T, cut=False)


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
@pytest.mark.parametrize("kind", ["slow", "full"])
def test_state_of_a_long_decode(kind, dtype):
    B, H, HK, T = 2, 4, 2, 1024
    p = {n: (x.to(dtype) if n != "s0" else x) for n, x in long_problem(kind, B, T, H, HK).items()}
    s = p["s0"].clone()
    for t in range(T):
        gw.gated_delta_decode_step(*[p[n][:, t].contiguous() for n in ("q", "k", "v", "omega", "beta")], s, scale=SCALE)
    _, want = ref.prefill(*[a.double() for a in args(p)], scale=SCALE)
    assert off(s, want) <= tolerance(kind, T, cut=False)
