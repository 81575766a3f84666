"""Arguments that must be tensors in the gate's, the norm's and the product's calls, since their types and shapes say what
is to be done: raw pointers and None are refused by name."""
import pytest
import torch

import combine_route_histogram_amd as mdc

BF = torch.bfloat16


@pytest.mark.parametrize("bad", [None, 4096])
def test_gate_needs_its_logits(bad):
    with pytest.raises(ValueError, match="logits must be a tensor"):
        mdc.mdc_gate(mdc.Shape(1, 0, 4, 64, 2, 8, 0), bad, None, torch.zeros((4, 2), dtype=torch.int32),
                     torch.zeros((4, 2)))


@pytest.mark.parametrize("name", ["x", "weight", "residual", "residual_out", "q"])
def test_norm_needs_the_tensors_that_carry_a_type(name):
    args = dict(x=torch.zeros((2, 64), dtype=BF), weight=torch.zeros(64, dtype=BF), y=torch.zeros((2, 64), dtype=BF))
    with pytest.raises(ValueError, match=f"{name} must be a tensor"):
        mdc.mdc_add_rms_norm(**{**args, name: 4096})
    if name in ("x", "weight"):
        with pytest.raises(ValueError, match=f"{name} must be a tensor"):
            mdc.mdc_add_rms_norm(**{**args, name: None})


@pytest.mark.parametrize("name", ["a", "w"])
@pytest.mark.parametrize("bad", [None, 4096])
def test_product_needs_the_tensors_that_carry_its_sizes(name, bad):
    f8 = torch.float8_e4m3fn
    args = dict(a=torch.zeros((4, 128)).to(f8), a_scale=torch.zeros((4, 1)), expert_token_nums=None,
                w=torch.zeros((8, 128)).to(f8), w_scale=torch.zeros((1, 1)), y=torch.zeros((4, 8), dtype=BF))
    with pytest.raises(ValueError, match=f"{name} must be a tensor"):
        mdc.mdc_gmm_fp8(**{**args, name: bad})
