"""Measured cases of the gated delta rule and of group norm with an activation.

The gated delta rule (per batch row and value head, state S of 64 key rows x 64 value
columns, w_t = exp(-exp(omega_t)) one decay per head and token, b_t the write strength):

    e_t = v_t - w_t S_{t-1}^T k_t
    S_t = w_t S_{t-1} + b_t k_t e_t^T
    y_t = scale S_t^T q_t

Group norm with an activation (x [N, L, C], channels last, one mean and variance for each n
and group of C / groups channels, over all L positions):

    z = (x - mean) / sqrt(var + eps) * gamma + beta
    y = act(z), or z * act(gate) with a gate

``run`` computes an operator in elementary torch operations where ``own`` is false, and by
the library's entry points where it is true; ``exact`` gives the same outputs in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

D = 64          # head size
CHUNK = 64      # tokens a chunk in the plain form
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the smallest prefill: a two-head layer over one chunk of tokens in fp32, where only
        # the call's latency counts
        dict(name="prefill tiny", op="prefill", B=1, T=64, H=2, HK=2, dtype="f32", decay="usual", state=False),
        # one layer of a 1.5B-class model over a training-size batch
        dict(name="prefill layer", op="prefill", B=8, T=4096, H=32, HK=32, dtype="bf16", decay="usual", state=True),
        # one long document, queries and keys shared by four value heads each, a ragged end
        dict(name="prefill long shared", op="prefill", B=1, T=65531, H=64, HK=16, dtype="bf16", decay="slow", state=True),
        # a single request generating
        dict(name="decode one", op="decode", B=1, H=32, HK=32, dtype="bf16", decay="usual"),
        # a full serving batch generating
        dict(name="decode batch", op="decode", B=256, H=32, HK=32, dtype="bf16", decay="usual"),
        # a gradient check's size: fp32, ragged, shared keys, strong decays among weak ones
        dict(name="backward small", op="backward", B=2, T=333, H=4, HK=2, dtype="f32", decay="extreme", state=True),
        # the training step of one layer
        dict(name="backward layer", op="backward", B=8, T=4096, H=32, HK=32, dtype="bf16", decay="usual", state=True),
        # a serving batch's output stage: each token's heads normalised, gated by SiLU
        dict(name="norm rows decode", op="norm", N=256, L=1, C=2048, groups=32, dtype="bf16", act="silu", gate=True),
        # the same stage over a training-size batch
        dict(name="norm rows layer", op="norm", N=32768, L=1, C=2048, groups=32, dtype="bf16", act="silu", gate=True),
        # statistics over positions too, odd lengths and channels: ten channels a group
        dict(name="norm positions", op="norm", N=8, L=4093, C=320, groups=32, dtype="bf16", act="silu", gate=False),
        # the output stage's gradient in training
        dict(name="norm rows backward", op="norm_backward", N=32768, L=1, C=2048, groups=32, dtype="bf16", act="silu", gate=True),
        # the gradient over positions, fp32, odd sizes
        dict(name="norm positions backward", op="norm_backward", N=3, L=1021, C=200, groups=8, dtype="f32", act="silu", gate=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "backward", "backward", "norm", "norm_backward"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("prefill", "decode", "backward"):
        HK = _log(rng, 1, 32)
        H = HK * rng.choice([1, 1, 2, 4])
        if op == "decode":
            return dict(op=op, B=max(1, min(_log(rng, 1, 512), 8192 // H)), H=H, HK=HK, dtype=dtype,
                        decay=rng.choice(["usual", "slow", "extreme"]))
        T = _log(rng, 1, 16384 if op == "prefill" else 6000)
        most = 4_000_000 if op == "prefill" else 1_000_000     # token-heads, below the largest listed
        B = max(1, min(_log(rng, 1, 16), most // (T * H)))
        if B * T * H > most:
            T = most // (B * H)
        return dict(op=op, B=B, T=T, H=H, HK=HK, dtype=dtype,
                    decay=rng.choice(["usual", "slow", "extreme"]), state=rng.random() < 0.7)
    groups = rng.choice([1, 2, 4, 8, 16, 32, 40])
    per = rng.choice([64, 64, 128, 1, 3, 8, 10, 25, 40, 96])
    C = groups * per
    rows = _log(rng, 1, min(60_000_000 // C, 40_000))
    L = 1 if rng.random() < 0.5 else _log(rng, 2, max(2, min(rows, 8192)))
    return dict(op=op, N=max(1, rows // L), L=L, C=C, groups=groups, dtype=dtype,
                act=rng.choice(["silu", "silu", "none"]), gate=rng.random() < 0.5)


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _omega(shape, decay, g):
    u = torch.rand(shape, generator=g, device="cuda")
    if decay == "usual":
        return -6.0 + 7.0 * u                     # w from 0.066 to 0.9975
    if decay == "slow":
        return -8.0 + 8.0 * u
    # strong decays (down to exp(-55)) on one token in eight, weak ones on the others
    strong = torch.rand(shape, generator=g, device="cuda") < 0.125
    return torch.where(strong, 2.0 + 2.0 * u, -8.0 + 4.0 * u)


def _unit(shape, g, dt):
    # keys and queries as a layer forms them: an activation, then unit length
    x = torch.nn.functional.silu(torch.randn(shape, generator=g, device="cuda"))
    return (x * torch.rsqrt(x.square().sum(-1, keepdim=True) + 1e-12)).to(dt)


def prepare(case, seed):
    g = _generator(seed)
    dt = DTYPES[case["dtype"]]
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    s = dict(case)
    if case["op"] in ("prefill", "decode", "backward"):
        B, H, HK = case["B"], case["H"], case["HK"]
        lead = (B,) if case["op"] == "decode" else (B, case["T"])
        s.update(q=_unit((*lead, HK, D), g, dt), k=_unit((*lead, HK, D), g, dt), v=rand(*lead, H, D).to(dt),
                 omega=_omega((*lead, H), case["decay"], g).to(dt), beta=torch.sigmoid(rand(*lead, H)).to(dt),
                 scale=D ** -0.5)
        s["s0"] = 0.1 * rand(B, H, D, D) if case.get("state", True) else None
        if case["op"] == "backward":
            s["dy"] = rand(*lead, H, D).to(dt)
            s["ds"] = 0.1 * rand(B, H, D, D) if case["state"] else None
        return s
    N, L, C = case["N"], case["L"], case["C"]
    s.update(x=(0.5 + 1.5 * rand(N, L, C)).to(dt), gamma=1.0 + 0.2 * rand(C), beta=0.1 * rand(C), eps=64e-5,
             gate=rand(N, L, C).to(dt) if case["gate"] else None)
    if case["op"] == "norm_backward":
        s["dy"] = rand(N, L, C).to(dt)
    return s


# ------------------------------------------------------------------ the gated delta rule, plain

def _chunks(x, T, fill=0.0):
    """[B, T, H, ...] -> [B, H, chunks, CHUNK, ...] fp32, the last chunk filled up."""
    n = -(-T // CHUNK) * CHUNK - T
    x = x.float()
    if n:
        x = torch.cat([x, x.new_full((x.shape[0], n, *x.shape[2:]), fill)], 1)
    return x.unflatten(1, (-1, CHUNK)).movedim(3, 1).contiguous()


def _tokens(x, T):
    return x.movedim(1, 3).flatten(1, 2)[:, :T]


def _inverse(a):
    """(I + a)^-1 of strictly lower triangular a, from blocks of one up: the lower left block of
    twice the size is -T22 a21 T11."""
    n = a.shape[-1]
    t = torch.eye(n, device=a.device).expand_as(a).clone()
    m = 1
    while m < n:
        blocks = n // (2 * m)
        i = torch.arange(blocks, device=a.device) * 2 * m
        lo, hi = (i[:, None] + torch.arange(m, device=a.device)), (i[:, None] + m + torch.arange(m, device=a.device))
        at = lambda x, r, c: x[..., r[:, :, None], c[:, None, :]]  # noqa: E731
        t[..., hi[:, :, None], lo[:, None, :]] = -(at(t, hi, hi) @ at(a, hi, lo) @ at(t, lo, lo))
        m *= 2
    return t


def _terms(s):
    T = s["q"].shape[1]
    r = s["H"] // s["HK"]
    heads = lambda x: x.repeat_interleave(r, 2) if r > 1 else x  # noqa: E731
    q, k, v = _chunks(heads(s["q"]), T), _chunks(heads(s["k"]), T), _chunks(s["v"], T)
    beta = _chunks(s["beta"], T)[..., None]
    lw = torch.cumsum(-torch.exp(_chunks(s["omega"], T, -math.inf).double()), -1)
    low = torch.tril(torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device))
    decay = torch.where(low, torch.exp((lw[..., :, None] - lw[..., None, :]).clamp(max=0.0)), 0.0).float()
    g = torch.exp(lw)[..., None].float()
    to_end = torch.exp(lw[..., -1:] - lw)[..., None].float()
    m = torch.tril(k @ k.mT * decay, -1)
    p = s["scale"] * (q @ k.mT) * decay
    t = _inverse(m * beta.mT)
    return dict(q=q, k=k, v=v, beta=beta, decay=decay, g=g, to_end=to_end, m=m, p=p, t=t, low=low, T=T)


def _states(c, s0):
    u, w = c["t"] @ c["v"], c["t"] @ (c["g"] * c["k"])
    kt = (c["to_end"] * c["k"]).mT
    s = torch.zeros_like(u[:, :, 0]) if s0 is None else s0
    states, news = [], []
    for n in range(u.shape[2]):
        e = torch.baddbmm(u[:, :, n].flatten(0, 1), w[:, :, n].flatten(0, 1), s.flatten(0, 1), alpha=-1).view_as(s)
        vn = c["beta"][:, :, n] * e
        states.append(s)
        news.append(e)
        s = c["g"][:, :, n, -1:] * s + kt[:, :, n] @ vn
    return torch.stack(states, 2), torch.stack(news, 2), s


def _plain_prefill(s):
    c = _terms(s)
    states, e, last = _states(c, s["s0"])
    y = s["scale"] * c["g"] * (c["q"] @ states) + c["p"] @ (c["beta"] * e)
    return _tokens(y, c["T"]).to(s["q"].dtype).contiguous(), last


def _plain_decode(s):
    r = s["H"] // s["HK"]
    q, k = (x.float().repeat_interleave(r, 1) for x in (s["q"], s["k"]))
    S = s["s0"]
    S.mul_(torch.exp(-torch.exp(s["omega"].float()))[..., None, None])
    e = s["v"].float() - (k[..., None] * S).sum(-2)
    S.add_((s["beta"].float()[..., None] * k)[..., None] * e[..., None, :])
    return (s["scale"] * (q[..., None] * S).sum(-2)).to(s["q"].dtype), S


def _plain_backward(s):
    c = _terms(s)
    T, scale = c["T"], s["scale"]
    states, e, last = _states(c, s["s0"])
    dy = _chunks(s["dy"], T)
    q, k, v, b, g = c["q"], c["k"], c["v"], c["beta"], c["g"]
    kt, vn = c["to_end"] * k, b * e
    # the state's gradient, chunk by chunk from the last
    x = c["p"].mT @ dy                                  # d vn without the state's part
    y0, w2 = c["t"].mT @ (b * x), c["t"].mT @ (b * kt)
    into = scale * (g * q).mT @ dy
    gk = (g * k).mT
    G = torch.zeros_like(last) if s["ds"] is None else s["ds"]
    grads = []
    for n in range(q.shape[2] - 1, -1, -1):
        grads.append(G)
        df = y0[:, :, n] + w2[:, :, n] @ G
        G = g[:, :, n, -1:] * G + into[:, :, n] - gk[:, :, n] @ df
    G0 = G
    G = torch.stack(grads[::-1], 2)
    dvn = x + kt @ G
    df = c["t"].mT @ (b * dvn)
    z = dvn - c["m"].mT @ df
    dp = scale * (dy @ vn.mT) * c["decay"]
    dm = torch.tril(-(df @ vn.mT) * c["decay"], -1)
    dq = scale * g * (dy @ states.mT) + dp @ k
    dk = dp.mT @ q + c["to_end"] * (vn @ G.mT) - g * (df @ states.mT) + (dm + dm.mT) @ k
    dbeta = (e * z).sum(-1)
    # the decay's gradient: w_t stands in every pair of a reader at t or after it and a source
    # before it, whether token or state (a difference of running sums would cancel where w_t is small)
    pairs = torch.tril((dy @ vn.mT) * c["p"] - (df @ vn.mT) * c["m"], -1)
    pairs = torch.tril(pairs.flip(-2).cumsum(-2).flip(-2), -1).sum(-1)
    reads = g[..., 0] * ((scale * q * (dy @ states.mT)).sum(-1) - (k * (df @ states.mT)).sum(-1))
    sources = (vn * (kt @ G)).sum(-1)
    dl = pairs + reads.flip(-1).cumsum(-1).flip(-1) + torch.nn.functional.pad(sources[..., :-1], (1, 0)).cumsum(-1)
    dl = dl + g[..., -1:, 0] * (G * states).sum((-1, -2))[..., None]
    domega = dl * -torch.exp(_chunks(s["omega"], T, -math.inf))
    dt = s["q"].dtype
    shared = lambda x: x.unflatten(2, (s["HK"], -1)).sum(3)  # noqa: E731
    out = [shared(_tokens(dq, T)), shared(_tokens(dk, T)), _tokens(df, T), _tokens(domega, T), _tokens(dbeta, T)]
    return [x.to(dt).contiguous() for x in out] + [G0]


# ------------------------------------------------------------------ group norm, plain

def _act(x, act):
    return x * torch.sigmoid(x) if act == "silu" else x


def _dact(x, act):
    if act != "silu":
        return torch.ones_like(x)
    t = torch.sigmoid(x)
    return t * (1 + x * (1 - t))


def _normal(s):
    N, L, C = s["x"].shape
    x = s["x"].float().view(N, L, s["groups"], -1)
    mean = x.mean((1, 3), keepdim=True)
    d = x - mean
    r = torch.rsqrt(d.square().mean((1, 3), keepdim=True) + s["eps"])
    return d * r, r


def _plain_norm(s):
    h, _ = _normal(s)
    z = h.flatten(2) * s["gamma"] + s["beta"]
    y = _act(z, s["act"]) if s["gate"] is None else z * _act(s["gate"].float(), s["act"])
    return y.to(s["x"].dtype)


def _plain_norm_backward(s):
    h, r = _normal(s)
    dt = s["x"].dtype
    z = h.flatten(2) * s["gamma"] + s["beta"]
    dy = s["dy"].float()
    dgate = None
    if s["gate"] is None:
        dz = dy * _dact(z, s["act"])
    else:
        gate = s["gate"].float()
        dz = dy * _act(gate, s["act"])
        dgate = (dy * z * _dact(gate, s["act"])).to(dt)
    dgamma, dbeta = (dz * h.flatten(2)).sum((0, 1)), dz.sum((0, 1))
    dh = (dz * s["gamma"]).view_as(h)
    dx = r * (dh - dh.mean((1, 3), keepdim=True) - h * (dh * h).mean((1, 3), keepdim=True))
    out = [dx.flatten(2).to(dt), dgamma, dbeta]
    return out if dgate is None else out + [dgate]


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["op"]
    if own:
        import linear_attention_rnn_finch_b200 as gw
        if op == "prefill":
            return gw.gated_delta_prefill(s["q"], s["k"], s["v"], s["omega"], s["beta"], s["s0"], scale=s["scale"])
        if op == "decode":
            y = gw.gated_delta_decode_step(s["q"], s["k"], s["v"], s["omega"], s["beta"], s["s0"], scale=s["scale"])
            return y, s["s0"]
        if op == "backward":
            return list(gw.gated_delta_backward(s["q"], s["k"], s["v"], s["omega"], s["beta"], s["s0"], s["dy"],
                                                s["ds"], scale=s["scale"]))
        if op == "norm":
            return gw.group_norm_act(s["x"], s["gamma"], s["beta"], s["eps"], groups=s["groups"], act=s["act"],
                                     gate=s["gate"])
        return [x for x in gw.group_norm_act_backward(s["x"], s["gamma"], s["beta"], s["eps"], s["dy"],
                                                      groups=s["groups"], act=s["act"], gate=s["gate"])
                if x is not None]
    if op == "prefill":
        return _plain_prefill(s)
    if op == "decode":
        return _plain_decode(s)
    if op == "backward":
        return _plain_backward(s)
    return _plain_norm(s) if op == "norm" else _plain_norm_backward(s)


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("norm", "norm_backward"):
        n, C = case["N"] * case["L"] * case["C"], case["C"]
        if case["op"] == "norm":
            return {"bytes": es * n * (3 if case["gate"] else 2) + 8 * C, "flops": n * (14 if case["gate"] else 12)}
        return {"bytes": es * n * (5 if case["gate"] else 3) + 16 * C, "flops": n * (30 if case["gate"] else 26)}
    B, T, H, HK = case["B"], case.get("T", 1), case["H"], case["HK"]
    th = B * T * H
    token = es * B * T * (2 * HK * D + H * D + 2 * H)          # q, k, v, omega, beta
    state = 4 * B * H * D * D
    has = 1 if case.get("state", True) else 0
    if case["op"] == "backward":
        return {"bytes": 2 * token + es * th * D + state * (2 * has + 1), "flops": 20 * D * D * th}
    return {"bytes": token + es * th * D + state * (1 + has), "flops": 7 * D * D * th}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The recurrences token by token, and their gradients by walking them back; the norm from
    its definition, its gradient through the quotient rule."""
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "norm_backward":
        with torch.enable_grad():
            leaves = [s[n].double().requires_grad_() for n in ("x", "gamma", "beta", "gate") if s[n] is not None]
            y = _exact_norm(dict(s, **dict(zip(("x", "gamma", "beta", "gate"), leaves))))
            return list(torch.autograd.grad(y, leaves, s["dy"].double()))
    r = case["H"] // case["HK"]
    q, k = (s[n].double().repeat_interleave(r, -2) for n in ("q", "k"))
    v, beta = s["v"].double(), s["beta"].double()
    rate = torch.exp(s["omega"].double())
    w = torch.exp(-rate)
    S = torch.zeros(v.shape[0], case["H"], D, D, dtype=torch.float64, device="cuda") if s["s0"] is None \
        else s["s0"].double()
    if case["op"] == "decode":
        q, k, v, beta, w = (x[:, None] for x in (q, k, v, beta, w))
    T = v.shape[1]

    def step(S, t):
        S = S * w[:, t, :, None, None]
        e = v[:, t] - torch.einsum("bhij,bhi->bhj", S, k[:, t])
        return S + torch.einsum("bhi,bhj->bhij", k[:, t] * beta[:, t, :, None], e), e

    if case["op"] != "backward":
        y = torch.empty_like(v)
        for t in range(T):
            S, _ = step(S, t)
            y[:, t] = s["scale"] * torch.einsum("bhij,bhi->bhj", S, q[:, t])
        return (y[:, 0] if case["op"] == "decode" else y), S
    dy = s["dy"].double()
    marks = []
    for t in range(T):
        if t % 64 == 0:
            marks.append(S)
        S, _ = step(S, t)
    G = torch.zeros_like(S) if s["ds"] is None else s["ds"].double()
    dq, dk, dv = (torch.empty_like(x) for x in (q, k, v))
    dw, dbeta = torch.empty_like(w), torch.empty_like(beta)
    for n in range(len(marks) - 1, -1, -1):
        S, held = marks[n], []
        for t in range(64 * n, min(T, 64 * n + 64)):
            after, e = step(S, t)
            held.append((S, e, after))
            S = after
        for t in range(min(T, 64 * n + 64) - 1, 64 * n - 1, -1):
            before, e, after = held[t - 64 * n]
            kt, bt = k[:, t], beta[:, t, :, None]
            dq[:, t] = s["scale"] * torch.einsum("bhij,bhj->bhi", after, dy[:, t])
            G = G + s["scale"] * torch.einsum("bhi,bhj->bhij", q[:, t], dy[:, t])
            ge = torch.einsum("bhij,bhj->bhi", G, e)
            gk = torch.einsum("bhij,bhi->bhj", G, kt)
            dbeta[:, t] = (kt * ge).sum(-1)
            de = bt * gk
            dv[:, t] = de
            sw = before * w[:, t, :, None, None]
            dk[:, t] = bt * ge - torch.einsum("bhij,bhj->bhi", sw, de)
            G = G - torch.einsum("bhi,bhj->bhij", kt, de)
            dw[:, t] = (G * before).sum((-1, -2))
            G = G * w[:, t, :, None, None]
    shared = lambda x: x.unflatten(2, (case["HK"], -1)).sum(3)  # noqa: E731
    return [shared(dq), shared(dk), dv, dw * w * -rate, dbeta, G]


def _exact_norm(s):
    x = s["x"].double().unflatten(2, (s["groups"], -1))
    var, mean = torch.var_mean(x, (1, 3), correction=0, keepdim=True)
    z = ((x - mean) / torch.sqrt(var + s["eps"])).flatten(2) * s["gamma"].double() + s["beta"].double()
    f = torch.nn.functional.silu if s["act"] == "silu" else (lambda t: t)
    return f(z) if s["gate"] is None else z * f(s["gate"].double())
