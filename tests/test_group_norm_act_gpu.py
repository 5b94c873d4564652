"""Group norm with an activation on the GPU against its definition in 64 bits: one position
(each token's heads) and several, group widths of one, odd, vector and beyond the registers,
channels that are no multiple of a vector, means far from zero, flat and outlying data, and the
gradients against autograd and differences.

Tolerances: the rounding to the output's type (eps / 2 of a value) plus the fp32 arithmetic,
against the largest value.  Statistics err by at most log-depth sums of differences from a
value of the data, about 32 x 2^-24 = 2e-6; with the division and activation 1e-5.  bf16 uses
the fast exponential and division, about 2^-21 more: 2e-5 covers both.  The gradients of gamma
and beta are sums over n and positions whose signs may leave a tenth: 1e-4.
"""
import ctypes

import pytest
import torch

import linear_attention_rnn_finch_b200 as gw
from linear_attention_rnn_finch_b200 import binding as bd
from tests import gated_delta_ref as ref
from tests.gated_delta_ref import c64, close

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
OWN, OWN_SUMS = 2e-5, 1e-4


def problem(seed, shape, dtype, gate, mean=0.5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)
    C = shape[-1]
    return dict(x=(mean + 1.5 * rn(*shape)).to(dtype), gamma=1 + 0.2 * rn(C), beta=0.1 * rn(C),
                gate=rn(*shape).to(dtype) if gate else None, dy=rn(*shape).to(dtype))


def check(p, groups, act, eps=1e-3, own=OWN, sums=OWN_SUMS):
    y = gw.group_norm_act(p["x"], p["gamma"], p["beta"], eps, groups=groups, act=act, gate=p["gate"])
    got = gw.group_norm_act_backward(p["x"], p["gamma"], p["beta"], eps, p["dy"], groups=groups,
                                     act=act, gate=p["gate"])
    leaves = [c64(p[n]).requires_grad_() for n in ("x", "gamma", "beta", "gate") if p[n] is not None]
    yo = ref.group_norm(*leaves[:3], eps, groups, act, *leaves[3:])
    close(y, yo, own, "y")
    want = torch.autograd.grad(yo, leaves, c64(p["dy"]))
    assert (got[3] is None) == (p["gate"] is None)
    for n, a, b in zip(("dx", "dgamma", "dbeta", "dgate"), got, want):
        close(a, b, sums if n in ("dgamma", "dbeta") else own, n)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("per", [1, 2, 3, 8, 10, 24, 33, 40, 64, 96, 128, 250, 256, 264, 300, 512, 520, 1024, 1032, 2048])
def test_rows_group_widths(per, dtype):
    check(problem(per, (37, 3 * per), dtype, True), 3, "silu")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("act", ["silu", "none"])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("N", [1, 5, 700])
def test_rows_forms(N, gate, act, dtype):
    check(problem(N, (N, 256), dtype, gate), 4, act)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L", [2, 3, 7, 8, 64, 129, 1021])
@pytest.mark.parametrize("C,groups", [(64, 1), (40, 8), (200, 8), (320, 32), (25, 5), (6, 6)])
def test_positions(L, C, groups, dtype):
    check(problem(L + C, (3, L, C), dtype, L % 2 == 0), groups, "silu" if C != 40 else "none")


@pytest.mark.parametrize("C,groups", [(2048, 32), (2056, 8), (4104, 2), (4104, 1), (2050, 10), (600, 2), (771, 3)])
def test_positions_wide(C, groups):
    """More channels than one tile, groups across its edge."""
    check(problem(C, (2, 19, C), BF16, True), groups, "silu")


def test_positions_many_axes_and_many_rows():
    check(problem(1, (2, 5, 7, 24), F32, True), 3, "silu")
    check(problem(2, (900, 2, 16), BF16, False), 2, "silu")
    check(problem(3, (1, 5000, 64), F32, False), 4, "none")


@pytest.mark.parametrize("shape,groups", [((40, 128), 2), ((2, 300, 32), 4)])
def test_mean_far_from_zero(shape, groups):
    """Mean 1000 at deviation 1.5: one step of the mean, 2^-24 x 1000 = 6e-5, over the deviation
    is 4e-5 of h, and the largest value is about 4: 1e-4 covers it.  Each dx, dgamma takes h."""
    check(problem(5, shape, F32, False, mean=1000.0), groups, "silu", own=1e-4, sums=1e-3)


@pytest.mark.parametrize("shape,groups", [((9, 64), 2), ((2, 130, 32), 4)])
@pytest.mark.parametrize("value", [0.0, 3.25])
def test_flat_groups(shape, groups, value):
    """No variance: h is 0, y the activation of beta."""
    p = problem(6, shape, F32, False)
    p["x"].fill_(value)
    y = gw.group_norm_act(p["x"], p["gamma"], p["beta"], 1e-5, groups=groups)
    want = p["beta"].double() / (1 + torch.exp(-p["beta"].double()))
    close(y, want.expand(shape).cpu(), 1e-6)


def test_first_position_outlies():
    """The value that differences are taken from is 1000 deviations away."""
    p = problem(7, (2, 4000, 32), F32, False, mean=0.0)
    p["x"][:, 0] = 1500.0
    check(p, 4, "none", sums=1e-3)   # dgamma: terms of h up to 60 that cancel


@pytest.mark.parametrize("shape,groups", [((33, 128), 2), ((3, 100, 40), 8)])
def test_gradients_against_differences(shape, groups):
    p = problem(8, shape, F32, True)
    got = gw.group_norm_act_backward(p["x"], p["gamma"], p["beta"], 1e-3, p["dy"], groups=groups, gate=p["gate"])
    a = [c64(p[n]) for n in ("x", "gamma", "beta", "gate")]
    g = torch.Generator().manual_seed(9)
    loss = lambda a: float((ref.group_norm(a[0], a[1], a[2], 1e-3, groups, "silu", a[3]) * c64(p["dy"])).sum())
    for i in range(4):
        d = torch.randn(a[i].shape, generator=g, dtype=torch.float64)
        up, down = list(a), list(a)
        up[i], down[i] = a[i] + 1e-4 * d, a[i] - 1e-4 * d
        want = (loss(up) - loss(down)) / 2e-4
        x = c64(got[i])
        assert abs(float((x * d).sum()) - want) <= OWN_SUMS * float(x.abs().max()) * float(d.norm()) + 1e-6 * abs(want)


def test_infinite_and_nan_rows_stay_their_own():
    """A row (or an n) with an infinity or a NaN leaves the others as they are."""
    for shape, groups in (((6, 128), 2), ((6, 50, 32), 4)):
        p = problem(10, shape, BF16, False)
        clean = gw.group_norm_act(p["x"], p["gamma"], p["beta"], groups=groups)
        p["x"][2].view(-1)[5] = float("inf")
        p["x"][4].view(-1)[9] = float("nan")
        y = gw.group_norm_act(p["x"], p["gamma"], p["beta"], groups=groups)
        keep = [0, 1, 3, 5]
        assert torch.equal(y[keep], clean[keep])
        assert bool(torch.isnan(y[4]).any())


@pytest.mark.parametrize("shape,groups", [((64, 512), 8), ((2, 300, 64), 4)])
def test_same_bits_on_a_stream_and_replayed(shape, groups):
    p = problem(11, shape, BF16, True)

    def calls():
        return [gw.group_norm_act(p["x"], p["gamma"], p["beta"], groups=groups, gate=p["gate"]),
                *gw.group_norm_act_backward(p["x"], p["gamma"], p["beta"], 1e-5, p["dy"], groups=groups, gate=p["gate"])]

    want = [x.clone() for x in calls()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls()
    for x in held:
        x.zero_()
    graph.replay()
    for x, y, z in zip(want, got, held):
        assert torch.equal(x, y) and torch.equal(x, z)


def test_empty():
    p = problem(12, (0, 64), BF16, False)
    assert gw.group_norm_act(p["x"], p["gamma"], p["beta"], groups=2).shape == (0, 64)
    for shape in ((0, 64), (3, 0, 64)):
        p = problem(12, shape, BF16, True)
        dx, dg, db, dgate = gw.group_norm_act_backward(p["x"], p["gamma"], p["beta"], 1e-5, p["dy"], groups=2, gate=p["gate"])
        assert dx.shape == shape and dgate.shape == shape
        assert bool((dg == 0).all()) and bool((db == 0).all())


def test_offsets_beyond_32_bits():
    """2.2e9 elements: the last rows are those of a call with them alone."""
    N, C = 1_100_000, 2048
    x = torch.empty(N, C, device=DEV, dtype=BF16).normal_(generator=torch.Generator(device=DEV).manual_seed(1))
    ga, be = torch.ones(C, device=DEV), torch.zeros(C, device=DEV)
    y = gw.group_norm_act(x, ga, be, groups=32)
    tail = gw.group_norm_act(x[-5:].contiguous(), ga, be, groups=32)
    assert torch.equal(y[-5:], tail)
    x3 = x.view(1, N, C)
    y = gw.group_norm_act(x3, ga, be, groups=32, act="none")
    cols = x3[0, :, :64].double()
    want = (x3[0, -3:, :64].double() - cols.mean()) / torch.sqrt(cols.var(correction=0) + 1e-5)
    close(y[0, -3:, :64].contiguous(), want.cpu(), OWN)


def test_refusals():
    p = problem(13, (4, 64), BF16, True)
    ok = dict(groups=2, gate=p["gate"])
    for kw in (dict(ok, groups=3), dict(ok, groups=0), dict(ok, act="gelu"), dict(ok, gate=p["gate"].float()),
               dict(ok, gate=p["gate"][:, :32])):
        with pytest.raises(ValueError):
            gw.group_norm_act(p["x"], p["gamma"], p["beta"], **kw)
    with pytest.raises(ValueError):
        gw.group_norm_act(p["x"].t(), p["gamma"], p["beta"], groups=2)
    with pytest.raises(ValueError):
        gw.group_norm_act(p["x"], p["gamma"].to(BF16), p["beta"], groups=2)
    with pytest.raises(ValueError):
        gw.group_norm_act(p["x"].half(), p["gamma"], p["beta"], groups=2)
    with pytest.raises(ValueError):
        gw.group_norm_act(p["x"].cpu(), p["gamma"], p["beta"], groups=2)
    with pytest.raises(gw.WkvError):
        gw.group_norm_act(p["x"], p["gamma"], p["beta"], 0.0, groups=2)
    with pytest.raises(gw.WkvError):
        gw.group_norm_act(p["x"], p["gamma"], p["beta"], float("nan"), groups=2)
    with pytest.raises(gw.WkvError):
        gw.group_norm_act(p["x"], p["gamma"], p["beta"], groups=2, y=p["x"])
    with pytest.raises(gw.WkvError):
        gw.group_norm_act_backward(p["x"], p["gamma"], p["beta"], 1e-5, p["dy"], groups=2,
                                   workspace=torch.empty(16, dtype=torch.uint8, device=DEV))


def test_entry_point_refusals():
    p = problem(14, (3, 10, 64), BF16, True)
    L = bd.load()
    vp = lambda t, off=0: None if t is None else ctypes.c_void_p(t.data_ptr() + off)
    y = torch.full_like(p["x"], 3.0)
    need = bd.group_norm_act_workspace_bytes(3, 10, 64, 2, BF16)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)

    def call(x=vp(p["x"]), eps=1e-5, act=1, yy=vp(y), sizes=(3, 10, 64, 2), io=1, w=vp(ws), n=need, gate=vp(p["gate"])):
        st = L.group_norm_act(x, vp(p["gamma"]), vp(p["beta"]), eps, act, gate, yy, *sizes, io, w, n, None)
        torch.cuda.synchronize()
        return st

    bad = bd.WKV_ERR_INVALID_ARG
    assert need > 0 and call(n=need - 1) == bd.WKV_ERR_WORKSPACE and call(w=None, n=0) == bd.WKV_ERR_WORKSPACE
    assert call(x=None) == bad and call(x=vp(p["x"], 2)) == bad and call(act=2) == bad and call(eps=-1.0) == bad
    assert call(sizes=(3, 10, 64, 5)) == bad and call(sizes=(3, 10, 0, 1)) == bad and call(sizes=(-1, 10, 64, 2)) == bad
    assert call(io=7) == bad and call(yy=vp(p["gate"])) == bad and call(w=vp(y)) == bad
    assert call(sizes=(1 << 40, 10, 64, 2)) == bd.WKV_ERR_UNSUPPORTED
    assert bool((y == 3.0).all())
    assert call() == bd.WKV_OK
    # a gate without a place for its gradient, and the other way round
    out = [torch.empty_like(p["x"]), torch.empty(64, device=DEV), torch.empty(64, device=DEV)]
    nb = bd.group_norm_act_workspace_bytes(3, 10, 64, 2, BF16, backward=True)
    wb = torch.empty(nb, dtype=torch.uint8, device=DEV)
    for gate, dgate in ((p["gate"], None), (None, torch.empty_like(p["x"]))):
        assert L.group_norm_act_backward(vp(p["x"]), vp(p["gamma"]), vp(p["beta"]), 1e-5, 1, vp(gate), vp(p["dy"]),
                                         *[vp(o) for o in out], vp(dgate), 3, 10, 64, 2, 1, vp(wb), nb, None) == bad
