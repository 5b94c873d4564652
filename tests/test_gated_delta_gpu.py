"""The gated delta rule on the GPU against the plain 64-bit recurrence: prefill, decode step and
gradients, over lengths around the chunk and tile edges, shared heads, decays from none to all,
write strengths of nothing, one and two, keys that are all alike, and a layer's run of them
together with the norm of its output stage."""
import ctypes

import pytest
import torch

import linear_attention_rnn_finch_b200 as gw
from linear_attention_rnn_finch_b200 import binding as bd
from tests import gated_delta_ref as ref
from tests.gated_delta_ref import OWN, OWN_GATES, c64, close

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16
SCALE = 0.125


def problem(seed, B, T, H, HK, dtype, decay="usual", state=True, alike=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device=DEV)
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    q, k = unit(rn(B, T, HK, 64)), unit(rn(B, T, HK, 64))
    if alike:
        k = unit(rn(B, 1, HK, 64)).expand(B, T, HK, 64) + 0.02 * rn(B, T, HK, 64)
        k = unit(k)
    om = {"usual": lambda: -6 + 7 * torch.rand((B, T, H), generator=g, device=DEV),
          "slow": lambda: -9 + 3 * torch.rand((B, T, H), generator=g, device=DEV),
          "strong": lambda: 2 + 2 * torch.rand((B, T, H), generator=g, device=DEV),
          "mixed": lambda: torch.where(torch.rand((B, T, H), generator=g, device=DEV) < 0.1, 4.0, -6.0),
          "ends": lambda: torch.tensor([-float("inf"), -60.0, -3.0, 30.0, float("inf")], device=DEV)[
              torch.randint(0, 5, (B, T, H), generator=g, device=DEV)]}[decay]()
    beta = torch.sigmoid(rn(B, T, H))
    p = dict(q=q, k=k, v=rn(B, T, H, 64), omega=om, beta=beta)
    p = {n: x.to(dtype).contiguous() for n, x in p.items()}
    p["s0"] = 0.3 * rn(B, H, 64, 64) if state else None
    return p


def args(p):
    return [p[n] for n in ("q", "k", "v", "omega", "beta", "s0")]


def check_prefill(p, dtype):
    y, s = gw.gated_delta_prefill(*args(p), scale=SCALE)
    yo, so = ref.prefill(*[c64(a) for a in args(p)], scale=SCALE)
    close(y, yo, OWN[dtype], "y")
    close(s, so, OWN[dtype], "state")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 63, 64, 65, 127, 129, 200, 333])
def test_prefill_lengths(T, dtype):
    check_prefill(problem(100 + T, 2, T, 3, 3, dtype), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,HK", [(1, 1, 1), (3, 4, 2), (2, 6, 1), (1, 40, 8), (5, 2, 2)])
def test_prefill_heads(B, H, HK, dtype):
    check_prefill(problem(7, B, 70, H, HK, dtype), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("decay", ["slow", "strong", "mixed", "ends"])
@pytest.mark.parametrize("state", [True, False])
def test_prefill_decays(decay, state, dtype):
    check_prefill(problem(11, 2, 190, 2, 2, dtype, decay, state), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("strength", [0.0, 0.5, 1.0, 2.0])
def test_prefill_keys_alike(strength, dtype):
    """Keys that nearly coincide: the chunk's triangular system is far from the identity."""
    p = problem(13, 1, 150, 2, 1, dtype, "slow", alike=True)
    p["beta"] = torch.full_like(p["beta"], strength)
    check_prefill(p, dtype)


def test_prefill_scale_zero_heads_and_empty():
    p = problem(17, 2, 40, 2, 2, BF16)
    y, _ = gw.gated_delta_prefill(*args(p), scale=0.0)
    assert bool((y == 0).all())
    for B, T, H in ((0, 5, 2), (2, 5, 0), (2, 0, 3)):
        z = lambda *s: torch.zeros(s, device=DEV, dtype=BF16)
        s0 = torch.randn(B, H, 64, 64, device=DEV)
        y, s = gw.gated_delta_prefill(z(B, T, H, 64), z(B, T, H, 64), z(B, T, H, 64), z(B, T, H), z(B, T, H), s0)
        assert y.shape == (B, T, H, 64)
        if T == 0:
            assert torch.equal(s, s0)
            _, s = gw.gated_delta_prefill(z(B, T, H, 64), z(B, T, H, 64), z(B, T, H, 64), z(B, T, H), z(B, T, H))
            assert bool((s == 0).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_padding_leaves_the_state(dtype):
    """beta = 0 with omega = -inf: the state behind the padding is the one before it."""
    p = problem(19, 2, 200, 2, 2, dtype)
    for t0 in (64, 101):
        cut = {n: (x[:, :t0].contiguous() if n != "s0" else x) for n, x in p.items()}
        pad = {n: (x.clone() if n != "s0" else x) for n, x in p.items()}
        pad["beta"][:, t0:] = 0
        pad["omega"][:, t0:] = -float("inf")
        y0, s0 = gw.gated_delta_prefill(*args(cut), scale=SCALE)
        y1, s1 = gw.gated_delta_prefill(*args(pad), scale=SCALE)
        close(s1, c64(s0), OWN[dtype], "state")
        close(y1[:, :t0].contiguous(), c64(y0), OWN[dtype], "y")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_state_in_place_and_in_pieces(dtype):
    p = problem(23, 2, 260, 3, 3, dtype)
    yo, so = ref.prefill(*[c64(a) for a in args(p)], scale=SCALE)
    s, ys = p["s0"].clone(), []
    for a, b in ((0, 64), (64, 65), (65, 200), (200, 260)):
        piece = [p[n][:, a:b].contiguous() for n in ("q", "k", "v", "omega", "beta")]
        y, out = gw.gated_delta_prefill(*piece, s, scale=SCALE, state_out=s)
        assert out is s
        ys.append(y)
    close(torch.cat(ys, 1), yo, OWN[dtype], "y")
    close(s, so, 2 * OWN[dtype], "state")   # four calls' states, each off by its own share
    y, none = gw.gated_delta_prefill(*args(p), scale=SCALE, want_state=False)
    assert none is None
    close(y, yo, OWN[dtype], "y")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,HK", [(1, 1, 1), (7, 3, 3), (4, 8, 2), (130, 5, 5)])
def test_decode_steps(B, H, HK, dtype):
    p = problem(29, B, 5, H, HK, dtype, "mixed")
    s = p["s0"].clone()
    yo, so = ref.prefill(*[c64(a) for a in args(p)], scale=SCALE)
    for t in range(5):
        y = gw.gated_delta_decode_step(*[p[n][:, t].contiguous() for n in ("q", "k", "v", "omega", "beta")], s, scale=SCALE)
        close(y, yo[:, t], OWN[dtype], f"y{t}")
    close(s, so, OWN[dtype], "state")


def test_decode_infinite_decays():
    p = problem(31, 2, 1, 4, 4, F32, "usual")
    for om in (-float("inf"), float("inf"), 90.0):
        p["omega"].fill_(om)
        s = p["s0"].clone()
        y = gw.gated_delta_decode_step(*[p[n][:, 0].contiguous() for n in ("q", "k", "v", "omega", "beta")], s, scale=SCALE)
        yo, so = ref.prefill(*[c64(a) for a in args(p)], scale=SCALE)
        close(y, yo[:, 0], OWN[F32], "y")
        close(s, so, OWN[F32], "state")


NAMES = ("dq", "dk", "dv", "domega", "dbeta", "dstate")


def check_backward(p, dtype, ds=True, own_scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(1)
    dy = torch.randn(p["v"].shape, generator=g, device=DEV).to(dtype)
    dS = 0.3 * torch.randn((p["v"].shape[0], p["v"].shape[2], 64, 64), generator=g, device=DEV) if ds else None
    got = gw.gated_delta_backward(*args(p), dy, dS, scale=SCALE)
    a = [c64(x) for x in args(p)]
    none = a[5] is None
    if none:
        a[5] = torch.zeros(got[5].shape, dtype=torch.float64)
    want = ref.gradients(a, c64(dy), c64(dS), scale=SCALE)
    for n, x, y in zip(NAMES, got, want):
        if y is None:
            y = torch.zeros(x.shape, dtype=torch.float64)
        y = torch.nan_to_num(y) if n == "domega" else y    # inf * 0 at omega = +inf: the limit is 0
        close(x, y, own_scale * (OWN_GATES if n in ("domega", "dbeta") else OWN)[dtype], n)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [1, 2, 17, 63, 64, 65, 129, 200])
def test_backward_lengths(T, dtype):
    check_backward(problem(200 + T, 2, T, 2, 2, dtype), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,HK", [(1, 1, 1), (2, 4, 2), (1, 6, 1), (3, 12, 4)])
def test_backward_shared_heads(B, H, HK, dtype):
    check_backward(problem(37, B, 90, H, HK, dtype), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("decay", ["slow", "strong", "mixed", "ends"])
def test_backward_decays(decay, dtype):
    check_backward(problem(41, 2, 150, 2, 2, dtype, decay, state=decay != "mixed"), dtype, ds=decay != "strong")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("strength", [0.0, 0.5, 1.0])
def test_backward_keys_alike(strength, dtype):
    p = problem(43, 1, 100, 2, 1, dtype, "slow", alike=True)
    p["beta"] = torch.full_like(p["beta"], strength)
    check_backward(p, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_backward_some_tokens_write_nothing(dtype):
    p = problem(47, 2, 130, 2, 2, dtype)
    p["beta"][:, ::3] = 0
    check_backward(p, dtype)


def test_backward_against_differences():
    """<gradient, direction> of every input against a central difference of the 64-bit loss,
    step 1e-4: truncation about 1e-8, far below the 1e-4 of the gradients' own error."""
    p = problem(53, 1, 100, 2, 1, F32)
    g = torch.Generator().manual_seed(2)
    dy, dS = torch.randn(1, 100, 2, 64, generator=g), 0.3 * torch.randn(1, 2, 64, 64, generator=g)
    got = gw.gated_delta_backward(*args(p), dy.to(DEV), dS.to(DEV), scale=SCALE)
    a = [c64(x) for x in args(p)]

    def loss(a):
        y, S = ref.prefill(*a, scale=SCALE)
        return (y * dy.double()).sum() + (S * dS.double()).sum()

    for i, n in enumerate(NAMES):
        d = torch.randn(a[i].shape, generator=g, dtype=torch.float64)
        up, down = list(a), list(a)
        up[i], down[i] = a[i] + 1e-4 * d, a[i] - 1e-4 * d
        want = float(loss(up) - loss(down)) / 2e-4
        x = c64(got[i])
        # each term's error is at most 1e-4 of the largest gradient, and their signs are random
        room = 1e-4 * float(x.abs().max()) * float(d.norm()) + 1e-6 * abs(want)
        assert abs(float((x * d).sum()) - want) <= room, (n, float((x * d).sum()), want)


def test_backward_without_state_gradient_and_empty():
    p = problem(59, 2, 40, 2, 2, BF16)
    dy = torch.randn_like(p["v"])
    a = gw.gated_delta_backward(*args(p), dy, scale=SCALE, want_dstate_in=False)
    b = gw.gated_delta_backward(*args(p), dy, scale=SCALE)
    assert a[5] is None
    for x, y in zip(a[:5], b[:5]):
        assert torch.equal(x, y)
    e = problem(59, 2, 0, 2, 2, BF16)
    dS = torch.randn(2, 2, 64, 64, device=DEV)
    out = gw.gated_delta_backward(*args(e), torch.empty_like(e["v"]), dS)
    assert torch.equal(out[5], dS)


@pytest.mark.parametrize("T", [50, 300])
def test_same_bits_twice_on_a_stream_and_replayed(T):
    p = problem(61, 2, T, 4, 2, BF16)
    dy = torch.randn_like(p["v"])

    def calls():
        y, s = gw.gated_delta_prefill(*args(p), scale=SCALE)
        return [y, s, *gw.gated_delta_backward(*args(p), dy, s, scale=SCALE)]

    want = [x.clone() for x in calls()]
    for x, y in zip(want, calls()):
        assert torch.equal(x, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = calls()
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip(want, got):
        assert torch.equal(x, y)
    # two captures with workspaces of their own, replayed in turn
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = calls()
        graphs.append((g, outs))
    for g, outs in graphs:
        for x in outs:
            x.zero_()
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    for _, outs in graphs:
        for x, y in zip(want, outs):
            assert torch.equal(x, y)


def test_two_streams_at_once():
    ps = [problem(67 + i, 2, 700, 8, 8, BF16) for i in range(2)]
    want = [gw.gated_delta_prefill(*args(p), scale=SCALE) for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = []
    for p, st in zip(ps, streams):
        with torch.cuda.stream(st):
            got.append(gw.gated_delta_prefill(*args(p), scale=SCALE))
    torch.cuda.synchronize()
    for (y, s), (yo, so) in zip(got, want):
        assert torch.equal(y, yo) and torch.equal(s, so)


def test_offsets_beyond_32_bits():
    """B 2, T 264,000, H 64: v has 2.16e9 elements.  A head's results are those of a call with
    that head alone, where it is computed the same way (one that splits sequences when there
    are few heads differs in rounding)."""
    B, T, H = 2, 264_000, 64
    g = torch.Generator(device=DEV).manual_seed(3)
    v = torch.empty(B, T, H, 64, device=DEV, dtype=BF16).normal_(generator=g)
    k = torch.empty(B, T, 1, 64, device=DEV, dtype=BF16).normal_(0, 0.125, generator=g)
    om = torch.empty(B, T, H, device=DEV, dtype=BF16).uniform_(-6, 0, generator=g)
    be = torch.empty(B, T, H, device=DEV, dtype=BF16).uniform_(0, 1, generator=g)
    y, s = gw.gated_delta_prefill(k, k, v, om, be, scale=SCALE)
    for b, h in ((0, 0), (1, 63)):
        one = lambda x: x[b:b + 1, :, h:h + 1].contiguous()
        kk = k[b:b + 1].contiguous()
        y1, s1 = gw.gated_delta_prefill(kk, kk, one(v), one(om), one(be), scale=SCALE)
        close(y[b:b + 1, :, h:h + 1], c64(y1), OWN[BF16], "y")
        close(s[b:b + 1, h:h + 1], c64(s1), OWN[BF16], "state")


# ------------------------------------------------------------------ a layer

def test_layer_prefill_then_decode():
    """A prompt through prefill and the gated norm, then tokens one by one from its state."""
    B, T, H, HK, more = 2, 130, 4, 2, 6
    p = problem(71, B, T + more, H, HK, BF16)
    g = torch.Generator(device=DEV).manual_seed(5)
    gate = torch.randn((B, T + more, H * 64), generator=g, device=DEV).to(BF16)
    gamma = 1 + 0.2 * torch.randn(H * 64, generator=g, device=DEV)
    beta = 0.1 * torch.randn(H * 64, generator=g, device=DEV)
    first = [p[n][:, :T].contiguous() for n in ("q", "k", "v", "omega", "beta")]
    y, s = gw.gated_delta_prefill(*first, p["s0"], scale=SCALE)
    outs = [gw.group_norm_act(y.view(B * T, H * 64), gamma, beta, 1e-5, groups=H,
                              gate=gate[:, :T].reshape(B * T, H * 64)).view(B, T, H * 64)]
    raw = [y]
    for t in range(T, T + more):
        y = gw.gated_delta_decode_step(*[p[n][:, t].contiguous() for n in ("q", "k", "v", "omega", "beta")], s, scale=SCALE)
        raw.append(y[:, None])
        outs.append(gw.group_norm_act(y.view(B, H * 64), gamma, beta, 1e-5, groups=H,
                                      gate=gate[:, t].contiguous())[:, None])
    yo, so = ref.prefill(*[c64(a) for a in args(p)], scale=SCALE)
    raw, out = torch.cat(raw, 1), torch.cat(outs, 1)
    close(raw, yo, OWN[BF16], "y")
    close(s, so, OWN[BF16], "state")
    # the norm of the y that was stored
    want = ref.group_norm(c64(raw).view(-1, H * 64), c64(gamma), c64(beta), 1e-5, H, "silu",
                          c64(gate).view(-1, H * 64)).view(B, T + more, H * 64)
    close(out, want, OWN[BF16], "out")


def test_layer_gradients():
    """The norm's gradient handed on to the recurrence's, fp32, against autograd of both."""
    B, T, H, HK = 2, 100, 4, 2
    p = problem(73, B, T, H, HK, F32)
    g = torch.Generator(device=DEV).manual_seed(6)
    gate = torch.randn((B * T, H * 64), generator=g, device=DEV)
    gamma = 1 + 0.2 * torch.randn(H * 64, generator=g, device=DEV)
    beta = 0.1 * torch.randn(H * 64, generator=g, device=DEV)
    dout = torch.randn((B * T, H * 64), generator=g, device=DEV)
    y, _ = gw.gated_delta_prefill(*args(p), scale=SCALE)
    dy, dgamma, dbeta, dgate = gw.group_norm_act_backward(y.view(B * T, H * 64), gamma, beta, 1e-2,
                                                          dout, groups=H, gate=gate)
    got = gw.gated_delta_backward(*args(p), dy.view(B, T, H, 64), scale=SCALE)
    leaves = [c64(a).requires_grad_() for a in (*args(p), gamma, beta, gate)]
    yo, _ = ref.prefill(*leaves[:6], scale=SCALE)
    out = ref.group_norm(yo.reshape(B * T, H * 64), leaves[6], leaves[7], 1e-2, H, "silu", leaves[8])
    want = torch.autograd.grad(out, leaves, c64(dout))
    # y's error (3e-5 of its largest) over the norm's divisor sqrt(var + 0.01) >= 0.1, against
    # y's largest of about 3: ten times the single operators' own
    for n, x, w in zip((*NAMES, "dgamma", "dbeta", "dgate"), (*got, dgamma, dbeta, dgate), want):
        close(x, w, 10 * OWN_GATES[F32], n)


# ------------------------------------------------------------------ refusals

def test_binding_refusals():
    p = problem(79, 2, 20, 4, 2, BF16)
    a = args(p)

    def bad(i, x, err=ValueError):
        b = list(a)
        b[i] = x
        with pytest.raises(err):
            gw.gated_delta_prefill(*b)

    bad(0, a[0].float())
    bad(1, a[1][:, :, :1].contiguous())
    bad(2, a[2][:, :, :3].contiguous())          # 3 value heads over 2 key heads
    bad(2, a[2].transpose(1, 2))
    bad(3, a[3].float())
    bad(4, a[4][:, :10].contiguous())
    bad(5, a[5].to(BF16))
    bad(0, a[0].cpu())
    bad(1, a[1].cpu())
    bad(0, None, TypeError)
    half = [x.half() if x is not None and x.dtype == BF16 else x for x in a]
    with pytest.raises(ValueError):
        gw.gated_delta_prefill(*half)
    with pytest.raises(gw.WkvError):
        gw.gated_delta_prefill(*a, scale=float("nan"))
    with pytest.raises(gw.WkvError):
        gw.gated_delta_prefill(*a, y=p["v"])     # y over an input
    with pytest.raises(gw.WkvError):
        gw.gated_delta_backward(*a, p["v"], workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        gw.gated_delta_decode_step(*a[:5], a[5])


def vp(t, off=0):
    return None if t is None else ctypes.c_void_p(t.data_ptr() + off)


def test_entry_point_refusals_touch_nothing():
    p = problem(83, 2, 20, 4, 2, BF16)
    L = bd.load()
    y = torch.full_like(p["v"], 3.0)
    s = torch.full_like(p["s0"], 7.0)
    need = bd.gated_delta_prefill_workspace_bytes(2, 20, 4, 2, 64, BF16)
    ws = bd.new_workspace(max(need, 16), DEV)

    def call(q=vp(p["q"]), k=vp(p["k"]), yy=vp(y), so=vp(s), si=vp(p["s0"]), sizes=(2, 20, 4, 2, 64), io=1, scale=1.0,
             om=vp(p["omega"])):
        st = L.gated_delta_prefill(q, k, vp(p["v"]), om, vp(p["beta"]), scale, si, so, yy,
                                   *sizes, io, vp(ws), ws.numel(), None)
        torch.cuda.synchronize()
        return st

    bad, unsup = bd.WKV_ERR_INVALID_ARG, bd.WKV_ERR_UNSUPPORTED
    assert call(q=None) == bad
    assert call(q=vp(p["q"], 2)) == bad
    assert call(k=vp(p["k"].cpu().pin_memory())) == bad
    assert call(yy=vp(p["v"])) == bad
    assert call(yy=None) == bad
    assert call(so=vp(p["s0"], 16)) == bad
    assert call(so=vp(y)) == bad
    assert call(om=vp(p["omega"], 1)) == bad
    assert call(sizes=(2, 20, 4, 3, 64)) == bad
    assert call(sizes=(2, 20, 4, 0, 64)) == bad
    assert call(sizes=(-1, 20, 4, 2, 64)) == bad
    assert call(sizes=(2, 20, 4, 2, 128)) == unsup
    assert call(sizes=(2, 2_000_000_000, 100, 2, 64)) == unsup
    assert call(io=2) == bad
    assert call(scale=float("inf")) == bad
    assert bool((y == 3.0).all()) and bool((s == 7.0).all())
    assert call() == bd.WKV_OK
    assert not bool((y == 3.0).all())


def test_backward_entry_point_refusals(monkeypatch):
    p = problem(89, 1, 20, 2, 2, F32)
    L = bd.load()
    outs = [torch.full_like(p[n], 3.0) for n in ("q", "k", "v", "omega", "beta")] + [torch.full_like(p["s0"], 3.0)]
    dy = torch.randn_like(p["v"])
    need = bd.gated_delta_backward_workspace_bytes(1, 20, 2, 2, 64, F32)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)

    def call(o=outs, w=ws, n=need):
        st = L.gated_delta_backward(*[vp(a) for a in args(p)[:5]], 1.0, vp(p["s0"]), vp(dy), None,
                                    *[vp(x) for x in o], 1, 20, 2, 2, 64, 0, vp(w), n, None)
        torch.cuda.synchronize()
        return st

    assert call(n=need - 1) == bd.WKV_ERR_WORKSPACE
    assert call(w=None, n=0) == bd.WKV_ERR_WORKSPACE
    assert call(o=[outs[1], *outs[1:]]) == bd.WKV_ERR_INVALID_ARG       # dq over dk
    assert call(o=[p["q"], *outs[1:]]) == bd.WKV_ERR_INVALID_ARG
    assert call(o=[*outs[:5], p["s0"]]) == bd.WKV_ERR_INVALID_ARG
    assert call(o=[None, *outs[1:]]) == bd.WKV_ERR_INVALID_ARG
    assert call(w=outs[2], n=need) in (bd.WKV_ERR_INVALID_ARG,)
    monkeypatch.setenv("GOLDWKV_FAULT", "launch")
    assert call() == bd.WKV_ERR_CUDA
    monkeypatch.delenv("GOLDWKV_FAULT")
    assert all(bool((x == 3.0).all()) for x in outs)
    assert call() == bd.WKV_OK
