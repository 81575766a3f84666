"""The expert layer of no tokens: what has no elements has no address, and the call is a success that does nothing."""
import ctypes

import pytest
import torch

import combine_route_histogram_amd as mdc

GATE = dict(dtype=mdc.MDC_DTYPE_FP32, score=mdc.MDC_GATE_SOFTMAX, groups=1, topk_groups=1, group_top=1, renormalise=1,
            scale=1.0)
EMPTY = mdc.Shape(world=1, rank=0, bs=0, hidden=512, topk=4, num_experts=32, capacity=0)
GPU = pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")
BOTH = pytest.mark.parametrize("name", ["mdc_moe", "mdc_moe_fp8"])


@BOTH
def test_no_tokens_with_a_gate(name):
    fn, none, some = getattr(mdc._lib, name), ctypes.c_void_p(None), ctypes.c_void_p(1 << 20)

    def call(gate, logits=none, ids=none, scales=none):
        return fn(EMPTY.c(), gate and mdc.mdc_gate_params(**gate), 512, none, logits, none, ids, scales, none, some, some, some,
                  some, none, none, none, some, 1 << 30, None)

    assert call(GATE) == mdc.MDC_OK            # logits of no tokens
    assert call(GATE, logits=some) == mdc.MDC_OK
    assert call(None) == mdc.MDC_OK and call(None, ids=some, scales=some) == mdc.MDC_OK
    assert call({**GATE, "groups": 5}) == mdc.MDC_ERR_INVALID   # the parameters are looked at all the same


@pytest.mark.gpu
@GPU
@BOTH
@pytest.mark.parametrize("routes", [False, True])
def test_no_tokens_through_the_binding(name, routes):
    e = lambda *s, d=torch.float32: torch.zeros(s, device="cuda").to(d)  # noqa: E731
    w, int8 = (torch.int8, True) if name == "mdc_moe" else (torch.float8_e4m3fn, False)
    s1, s2 = (e(32, 512), e(32, 512)) if int8 else (e(32, 4, 4), e(32, 4, 2))
    ws = torch.full((getattr(mdc, name + "_workspace")(EMPTY, 512),), 0x5A, dtype=torch.uint8, device="cuda")
    r = (e(0, 4, d=torch.int32), e(0, 4)) if routes else (None, None)
    getattr(mdc, name)(EMPTY, 512, e(0, 512, d=torch.bfloat16), e(0, 32), None, *r, e(32, 512, 512, d=w), s1,
                       e(32, 512, 256, d=w), s2, e(0, 512, d=torch.bfloat16), ws)
    torch.cuda.synchronize()
    assert (ws == 0x5A).all()


@pytest.mark.gpu
@GPU
def test_no_rows_through_the_binding():
    e = lambda *s, d=torch.float32: torch.zeros(s, device="cuda").to(d)  # noqa: E731
    bf, i8 = torch.bfloat16, torch.int8
    mdc.mdc_gmm_int8(e(0, 256, d=i8), e(0), e(2, d=torch.int64), e(2, 64, 256, d=i8), e(2, 64), e(0, 64, d=bf))
    for gate in (None, e(0, 256, d=bf), e(1, 256, d=bf), e(0, 1, d=bf)):
        mdc.mdc_block_rms_norm(e(0, 256, d=bf), e(256, d=bf), post_weight=e(256, d=bf), gate=gate, residual=e(0, 256),
                               residual_out=e(0, 256), y=e(0, 256, d=bf), q=e(0, 256, d=i8), q_scale=e(0))
    torch.cuda.synchronize()
