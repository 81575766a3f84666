"""Renormalised sigmoid weights where the chosen logits are far below zero: 1 / (1 + exp(-z)) leaves fp32 there, the
quotient by the sum does not."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tests.test_gpu_gate import check, run  # noqa: E402


def low_rows(T, n, dtype, seed):
    """Rows around -10 to -700: near each other, and with one or two logits well above the rest."""
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((T, n), generator=g)
    z += torch.tensor([-10.0, -80.0, -88.0, -95.0, -104.0, -200.0, -700.0])[torch.arange(T) % 7, None]
    z[::3, 1] += 60.0
    z[::5, 2] += 20.0
    return z.to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,n,k", [(1, 16, 4), (35, 64, 8), (33, 256, 8), (4101, 64, 16), (4097, 256, 6)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_low_logits_share_the_weight(T, n, k, dtype, with_bias):
    logits = low_rows(T, n, dtype, n + k)
    bias = 0.1 * torch.randn((n,), generator=torch.Generator().manual_seed(1)) if with_bias else None
    check(logits, bias, k, score="sigmoid", scale=2.5)
    check(logits, bias, k, score="sigmoid", groups=4, topk_groups=2, group_top=1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("low", [-80.0, -88.0, -95.0, -200.0, -700.0])
def test_equal_low_logits_get_equal_weights(low, dtype):
    _, w = run(torch.full((5, 16), low, dtype=dtype), None, 4, score="sigmoid")
    assert np.all(np.abs(w - 0.25) <= 2.0 ** -24)   # four equal addends, one quotient


@pytest.mark.parametrize("with_bias", [False, True])
def test_scores_that_are_zero_in_64_bits_weigh_nothing(with_bias):
    """exp(-z) passes 64 bits below z = -709.78: the score is 0 there, and a row of such scores has no weight."""
    logits = torch.full((6, 32), -3.4028234663852886e38)
    logits[1] = -720.0
    logits[2] = -709.5
    logits[3, ::2] = -709.0
    logits[3, 1::2] = -712.0
    logits[4, 3] = -5.0
    logits[5, 7] = 4.0
    bias = torch.linspace(0.5, 1.0, 32) if with_bias else None
    with np.errstate(over="ignore"):
        check(logits, bias, 8, score="sigmoid")
    _, w = run(logits, bias, 8, score="sigmoid")
    assert not w[:2].any() and np.allclose(w[2], 1 / 8)
