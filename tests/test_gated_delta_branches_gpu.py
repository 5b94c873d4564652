"""Gradients of the gated delta rule where the launches take another form: key heads and chunks that
fill the device, so that one block of threads walks the value heads of a key head (fp32), and
keys that are alike at write strengths up to two."""
import pytest
import torch

from tests.test_gated_delta_gpu import BF16, F32, check_backward, problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,T,H,HK", [(19, 130, 8, 4), (25, 101, 12, 3), (1, 1217, 16, 8)])
def test_shared_heads_that_fill_the_device(B, T, H, HK, dtype):
    assert H > HK and B * HK * -(-T // 64) >= 148 and T % 64
    check_backward(problem(600 + T, B, T, H, HK, dtype), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T", [100, 330])
@pytest.mark.parametrize("strength", [1.5, 2.0])
def test_keys_alike_at_strengths_up_to_two(strength, T, dtype):
    p = problem(610, 1, T, 2, 1, dtype, "slow", alike=True)
    p["beta"] = torch.full_like(p["beta"], strength)
    check_backward(p, dtype)
