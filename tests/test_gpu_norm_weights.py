"""Rows and weights whose product leaves fp32 where the normalised row times the weight does not."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tests.test_gpu_norm import BF, F16, F32, run_and_check  # noqa: E402


def tensors(rows, H, dtype, w_dtype, x_size, w_size, seed):
    g = torch.Generator().manual_seed(seed)
    x = (x_size * (0.5 + torch.rand((rows, H), generator=g)) * torch.where(torch.rand((rows, H), generator=g) < 0.5, -1., 1.))
    w = w_size * (0.5 + torch.rand((H,), generator=g))
    w[H // 2:] *= 2.0 ** -10   # runs of other sizes in the same row
    return x.to(dtype), None, w.to(w_dtype)


@pytest.mark.parametrize("quant", ["none", "int8", "fp8"])
@pytest.mark.parametrize("w_dtype", [BF, F32])
# 1e15 * 1e30 is above fp32's range; 1e-15 * 1e-28 and 1e-12 * 1e-30 are below it (of a row whose mean square is not)
@pytest.mark.parametrize("x_size,w_size", [(1e15, 1e30), (100.0, 1e37), (1e-15, 1e-28), (1e-12, 1e-30)])
@pytest.mark.parametrize("rows,H", [(3, 512), (2, 1160), (2, 9000)])
def test_products_outside_fp32(rows, H, x_size, w_size, w_dtype, quant):
    run_and_check(rows, H, BF, None, w_dtype, quant, True, tensors=tensors(rows, H, BF, w_dtype, x_size, w_size, H),
                  eps=0.0)


@pytest.mark.parametrize("quant", ["int8", "fp8"])
def test_products_outside_fp32_of_fp16_rows(quant):
    run_and_check(3, 512, F16, None, F32, quant, False, tensors=tensors(3, 512, F16, F32, 100.0, 1e37, 1))
