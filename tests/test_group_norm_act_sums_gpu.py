"""Group norm with an activation where a thread adds up many values: sets of lanes that walk
several rows, statistics over hundreds of positions behind an outlying first one, and parameter
gradients over hundreds of thousands of n."""
import pytest
import torch

import linear_attention_rnn_finch_b200 as gw
from tests.test_group_norm_act_gpu import BF16, DEV, F32, OWN, check, close, problem

pytestmark = pytest.mark.gpu


def most_streams(C, groups, ctas):
    """Rows that are walked at once: sets of lanes, of 256 / lanes a block, over the groups."""
    per = C // groups
    units = per // 8 if per % 8 == 0 else per
    lanes = min(32, 1 << (units - 1).bit_length())
    return -(-148 * ctas * (256 // lanes) // groups)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("act,gate", [("silu", True), ("silu", False), ("none", True), ("none", False)])
@pytest.mark.parametrize("groups,per,N", [(40, 64, 2500), (40, 24, 2500), (32, 1032, 301), (24, 10, 1999),
                                          (16, 100, 1403), (16, 40, 5003), (8, 520, 2503), (8, 300, 2503)])
def test_rows_walked_by_one_set(groups, per, N, act, gate, dtype):
    """More rows than are walked at once (8 blocks an SM forward, 3 in the gradient) and no
    multiple of them, so that some sets end a row early."""
    C = groups * per
    for ctas in (3, 8):
        streams = most_streams(C, groups, ctas)
        assert N > streams and N % streams
    check(problem(40 + per, (N, C), dtype, gate), groups, act)


def statistics_of_many(C, groups, own, fill):
    """y of [300, 1000, C], where a thread adds up 1000 positions, against 64 bits."""
    N, L = 300, 1000
    g = torch.Generator(device=DEV).manual_seed(7)
    x = torch.empty(N, L, C, device=DEV).normal_(0, 1.5, generator=g)
    fill(x)
    ga, be = torch.ones(C, device=DEV), torch.zeros(C, device=DEV)
    y = gw.group_norm_act(x, ga, be, 1e-3, groups=groups, act="none")
    for n in (0, N - 1):
        h = x[n].double().view(L, groups, -1)
        var, mean = torch.var_mean(h, (0, 2), correction=0, keepdim=True)
        want = ((h - mean) / torch.sqrt(var + 1e-3)).view(L, C)
        close(y[n], want.cpu(), own, f"y[{n}]")


@pytest.mark.parametrize("C,groups", [(2048, 32), (250, 10)])
@pytest.mark.parametrize("at", [0, 500])
def test_a_position_outlies_many(at, C, groups):
    """One position, the first, from whose value the others' differences start, or one amid them, is
    1000 deviations away: the same tolerance as for a few positions a thread."""
    statistics_of_many(C, groups, OWN, lambda x: x[:, at].fill_(1500.0))


@pytest.mark.parametrize("C,groups", [(2048, 2048), (250, 10)])
def test_mean_far_from_zero_over_many(C, groups):
    """Mean 1000 at deviation 1.5 joined 16 times: one step of the mean, 2^-24 x 1000 = 6e-5, over the
    deviation is 4e-5 of h, whose largest is above 4: 1e-4, as for few positions."""
    statistics_of_many(C, groups, 1e-4, lambda x: x.add_(1000.0))


@pytest.mark.parametrize("N,L", [(400_000, 2), (3000, 300)])
def test_parameter_gradients_of_many(N, L):
    """dbeta is the sum of N L values of one sign, dgamma that of as many products.  A row of partial
    sums holds at most 2 + 128 additions, eight rows and the warps' sums 3 + 32 more, each off by
    2^-25 on average with independent signs: under sqrt(165) 2^-25 = 3.8e-7 of the magnitudes; with
    what rounding takes from the running sum carried on it stays that however many there are.
    Rounding the result adds 2^-24, and the largest of 32 columns may be twice the average."""
    C, groups = 16, 2
    g = torch.Generator(device=DEV).manual_seed(N)
    x = torch.randn(N, L, C, generator=g, device=DEV)
    dy = 1 + torch.rand(N, L, C, generator=g, device=DEV)
    ga, be = torch.ones(C, device=DEV), torch.zeros(C, device=DEV)
    _, dgamma, dbeta, _ = gw.group_norm_act_backward(x, ga, be, 1e-3, dy, groups=groups, act="none")
    d = dy.double()
    h = x.double().view(N, L, groups, -1)
    var, mean = torch.var_mean(h, (1, 3), correction=0, keepdim=True)
    h = ((h - mean) / torch.sqrt(var + 1e-3)).view(N, L, C)
    for got, terms in ((dbeta, d), (dgamma, d * h)):
        off = (got.double() - terms.sum((0, 1))).abs() / terms.abs().sum((0, 1))
        assert float(off.max()) <= 9e-7, float(off.max())


@pytest.mark.parametrize("shape", [(3000, 2, 32), (70_000, 32)])
def test_infinite_gradients_stay_in_their_channel(shape):
    """dy infinite in one place of a channel: its dbeta is that infinity, wherever the place comes in the
    sum, and the other channels' sums are those without it."""
    p = problem(60, shape, F32, False)
    at = p["dy"].view(-1, 32)
    call = lambda: gw.group_norm_act_backward(p["x"], p["gamma"], p["beta"], 1e-3, p["dy"], groups=4, act="none")[1:3]
    clean = call()
    at[5, 3], at[2999, 20] = float("inf"), -float("inf")
    dgamma, dbeta = call()
    assert float(dbeta[3]) == float("inf") and float(dbeta[20]) == -float("inf")
    assert bool(torch.isinf(dgamma[[3, 20]]).all())
    keep = [c for c in range(32) if c not in (3, 20)]
    for got, want in zip((dgamma, dbeta), clean):
        assert torch.equal(got[keep], want[keep])
