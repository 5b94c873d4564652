"""Plain 64-bit forms of the gated delta rule and of group norm with an activation, on the CPU,
for the tests: the recurrences as they are defined, token by token, with torch's autograd for
their gradients.  Nothing here follows the chunked algebra of the kernels.

Tolerances.  A value rounded to type t is off by at most eps(t) / 2 of itself.  Besides that
rounding the kernels carry errors of their own arithmetic, bounded against the largest value of
the tensor:
  fp32 I/O: a sum of 64 products errs by at most 64 x 2^-24 = 3.8e-6 of the sum of their
    magnitudes; five such sums in a row, half of whose magnitudes may cancel: 3e-5.
  bf16 I/O: tensor-core operands are kept as two bf16 parts, 2^-17 = 7.6e-6 each; four of them
    in a row, a third of whose magnitudes may remain: 1e-4.
  domega and dbeta add up to 64 x 64 pairs in two levels of 64-term sums, (64 + 64) x 2^-24 =
    7.6e-6 of a sum of magnitudes of which signs may leave a tenth: 1e-4 with fp32 I/O; with
    bf16 I/O two more parts of 2^-17 a pair, a tenth left: 2e-4 + 1e-4 = 3e-4.
"""
from __future__ import annotations

import torch

OWN = {torch.float32: 3e-5, torch.bfloat16: 1e-4}
OWN_GATES = {torch.float32: 1e-4, torch.bfloat16: 3e-4}


def close(got, want, own, what=""):
    """|got - want| <= eps/2 |want| (the rounding to got's type) + own max|want|."""
    assert got.shape == want.shape, (what, got.shape, want.shape)
    g, w = got.detach().cpu().double(), want.detach().double()
    assert torch.isfinite(g).all(), f"{what}: not finite"
    if w.numel() == 0:
        return
    top = w.abs().max()
    room = torch.finfo(got.dtype).eps / 2 * w.abs() + own * (top if top > 0 else 1.0)
    off = (g - w).abs() - room
    assert off.max() <= 0, f"{what}: {float((g - w).abs().max()):.3g} off of {float(top):.3g}, {int((off > 0).sum())} values"


def c64(t):
    return None if t is None else t.detach().cpu().double()


def prefill(q, k, v, omega, beta, s0=None, scale=1.0):
    """q, k [B, T, HK, D], v [B, T, H, D], omega, beta [B, T, H] -> (y, state), differentiable."""
    B, T, H, D = v.shape
    r = H // q.shape[2] if q.shape[2] else 1
    q, k = q.repeat_interleave(r, 2), k.repeat_interleave(r, 2)
    w = torch.exp(-torch.exp(omega))
    S = torch.zeros(B, H, D, D, dtype=v.dtype) if s0 is None else s0
    ys = []
    for t in range(T):
        S = S * w[:, t, :, None, None]
        e = v[:, t] - torch.einsum("bhij,bhi->bhj", S, k[:, t])
        S = S + torch.einsum("bhi,bhj->bhij", k[:, t], beta[:, t, :, None] * e)
        ys.append(scale * torch.einsum("bhij,bhi->bhj", S, q[:, t]))
    y = torch.stack(ys, 1) if ys else v.new_zeros(B, 0, H, D)
    return y, S


def gradients(args, dy, ds, scale=1.0):
    """Gradients of prefill's inputs (None stays None) for dy and the final state's ds (or None)."""
    leaves = [None if a is None else a.clone().requires_grad_() for a in args]
    with torch.enable_grad():
        y, S = prefill(*leaves, scale=scale)
        loss = (y * dy).sum() + (0 if ds is None else (S * ds).sum())
    live = [a for a in leaves if a is not None]
    got = iter(torch.autograd.grad(loss, live, allow_unused=True))
    return [None if a is None else next(got) for a in leaves]


def group_norm(x, gamma, beta, eps, groups, act, gate=None):
    """x [N, ..., C] -> y, differentiable."""
    N, C = x.shape[0], x.shape[-1]
    h = x.reshape(N, -1, groups, C // groups)
    mean = h.mean((1, 3), keepdim=True)
    var = ((h - mean) ** 2).mean((1, 3), keepdim=True)
    z = ((h - mean) / torch.sqrt(var + eps)).reshape(x.shape) * gamma + beta
    f = (lambda t: t / (1 + torch.exp(-t))) if act == "silu" else (lambda t: t)
    return f(z) if gate is None else z * f(gate)
