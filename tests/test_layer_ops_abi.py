"""Argument checks of the int8 product, the norms around a block and the expert layer for a few tokens (no GPU needed: every
call returns before anything is enqueued), and closed forms of their oracles."""
import ctypes

import numpy as np
import pytest
import torch

import combine_route_histogram_amd as mdc
from oracle import ops64 as O

FAKE = 1 << 20
P = ctypes.c_void_p
NULL, INVALID, UNSUPPORTED = mdc.MDC_ERR_NULLPTR, mdc.MDC_ERR_INVALID, mdc.MDC_ERR_UNSUPPORTED


def gmm_status(A=64, L=4, n=64, k=128, dtype=mdc.MDC_DTYPE_BF16, a=FAKE, sa=FAKE, nums=FAKE, w=FAKE, sw=FAKE, y=FAKE):
    return mdc._lib.mdc_gmm_int8(A, L, n, k, dtype, P(a), P(sa), P(nums), P(w), P(sw), P(y), None)


@pytest.mark.parametrize("kw,want", [
    (dict(a=None), NULL), (dict(sa=None), NULL), (dict(nums=None), NULL), (dict(w=None), NULL), (dict(sw=None), NULL),
    (dict(y=None), NULL), (dict(A=-1), INVALID), (dict(L=0), INVALID), (dict(n=0), INVALID), (dict(n=60), INVALID),
    (dict(k=0), INVALID), (dict(k=136), INVALID), (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID),
    (dict(a=FAKE + 8), INVALID), (dict(w=FAKE + 8), INVALID), (dict(y=FAKE + 8), INVALID), (dict(sa=FAKE + 2), INVALID),
    (dict(sw=FAKE + 2), INVALID), (dict(nums=FAKE + 4), INVALID),
    (dict(L=2049), UNSUPPORTED), (dict(A=2 ** 31), UNSUPPORTED), (dict(n=1 << 16, k=1 << 15), UNSUPPORTED),
    (dict(n=8, k=1 << 17), UNSUPPORTED), (dict(A=2 ** 31 - 1, n=1 << 14, k=16), UNSUPPORTED),
    (dict(A=0, a=None, w=None, y=None), mdc.MDC_OK),
])
def test_gmm_int8_argument_checks(kw, want):
    assert gmm_status(**kw) == want


def block_status(x=FAKE, post=FAKE, gate=FAKE, res=FAKE, w=FAKE, res_out=FAKE, y=FAKE, q=None, s=None, params=True, **over):
    kw = dict(rows=4, gate_every=1, hidden=64, dtype=mdc.MDC_DTYPE_BF16, residual_dtype=mdc.MDC_DTYPE_BF16,
              weight_dtype=mdc.MDC_DTYPE_BF16, gate_dtype=mdc.MDC_DTYPE_BF16, gate_columns=64, gate_act=mdc.MDC_ACT_NONE,
              quant=mdc.MDC_QUANT_NONE, block_scale=1.0, residual_scale=1.0, post_eps=1e-6, eps=1e-6)
    kw.update(over)
    return mdc._lib.mdc_block_rms_norm(mdc.mdc_block_norm_params(**kw) if params else None, P(x), P(post), P(gate), P(res),
                                       P(w), P(res_out), P(y), P(q), P(s), None)


@pytest.mark.parametrize("kw,want", [
    (dict(params=False), NULL), (dict(x=None), NULL), (dict(w=None), NULL),                      # y without weight
    (dict(y=None, res_out=None), NULL), (dict(quant=mdc.MDC_QUANT_INT8), NULL), (dict(q=FAKE, s=FAKE), NULL),
    (dict(quant=mdc.MDC_QUANT_FP8, q=FAKE), NULL), (dict(s=FAKE), NULL),
    (dict(dtype=mdc.MDC_DTYPE_FP32), INVALID), (dict(residual_dtype=mdc.MDC_DTYPE_FP16), INVALID),
    (dict(weight_dtype=mdc.MDC_DTYPE_FP16), INVALID), (dict(gate_dtype=mdc.MDC_DTYPE_FP16), INVALID),
    (dict(quant=3), INVALID), (dict(gate_act=3), INVALID), (dict(gate_act=-1), INVALID), (dict(gate_columns=2), INVALID),
    (dict(gate_columns=0), INVALID), (dict(gate_every=0), INVALID), (dict(rows=-1), INVALID), (dict(hidden=0), INVALID),
    (dict(hidden=60), INVALID), (dict(eps=-1.0), INVALID), (dict(post_eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(block_scale=float("inf")), INVALID), (dict(residual_scale=float("nan")), INVALID),
    (dict(x=FAKE + 8), INVALID), (dict(post=FAKE + 8), INVALID), (dict(gate=FAKE + 8), INVALID), (dict(res=FAKE + 8), INVALID),
    (dict(w=FAKE + 8), INVALID), (dict(res_out=FAKE + 8), INVALID), (dict(y=FAKE + 8), INVALID),
    (dict(gate=FAKE + 1, gate_columns=1), INVALID), (dict(gate=FAKE + 2, gate_columns=1, gate_dtype=2), INVALID),
    (dict(quant=mdc.MDC_QUANT_FP8, q=FAKE + 4, s=FAKE), INVALID), (dict(quant=mdc.MDC_QUANT_FP8, q=FAKE, s=FAKE + 2), INVALID),
    (dict(hidden=32776, gate_columns=1), UNSUPPORTED), (dict(rows=2 ** 31), UNSUPPORTED),
    (dict(rows=0, x=None, w=None, y=None), mdc.MDC_OK),
])
def test_block_norm_argument_checks(kw, want):
    assert block_status(**kw) == want


MOE = mdc.Shape(world=4, rank=1, bs=8, hidden=512, topk=4, num_experts=32, capacity=0)
GATE = dict(dtype=mdc.MDC_DTYPE_FP32, score=mdc.MDC_GATE_SOFTMAX, groups=1, topk_groups=1, group_top=1, renormalise=1,
            scale=1.0)
NAMES = ["x", "logits", "bias", "ids", "scales", "mask", "w1", "w1s", "w2", "w2s", "shared", "ori", "out", "ws"]


def moe_status(fn, shape=MOE, inter=512, gate=None, bytes_=None, **over):
    need = 1 << 30
    v = {n: FAKE for n in NAMES}
    v.update(bias=None, mask=None, logits=FAKE if gate else None)
    v.update(over)
    pr = None if gate is None else mdc.mdc_gate_params(**gate)
    return fn(shape.c(), pr, inter, *[P(v[n]) for n in NAMES], need if bytes_ is None else bytes_, None)


@pytest.mark.parametrize("name", ["mdc_moe", "mdc_moe_fp8"])
def test_moe_argument_checks(name):
    fn, size = getattr(mdc._lib, name), getattr(mdc, name + "_workspace")
    shape = lambda **kw: mdc.Shape(**{**MOE.__dict__, **kw})  # noqa: E731
    need = size(MOE, 512)
    # status block, codes of x, g
    assert need >= mdc.MDC_STATUS_BYTES + 8 * 512 + 8 * 4 * 256 * 4
    for sh, inter, code in ((MOE, 0, INVALID), (MOE, 384, UNSUPPORTED), (shape(hidden=520), 512, UNSUPPORTED),
                            (shape(hidden=8320), 512, UNSUPPORTED), (shape(bs=33), 512, UNSUPPORTED),
                            (shape(num_experts=30), 512, INVALID), (shape(bs=-1), 512, INVALID),
                            (shape(hidden=8192), 1 << 18, UNSUPPORTED)):
        with pytest.raises(mdc.MdcError) as ei:
            size(sh, inter)
        assert ei.value.status == code
        assert moe_status(fn, sh, inter) == code
    for n in ("x", "w1", "w1s", "w2", "w2s", "out", "ws"):
        assert moe_status(fn, **{n: None}) == NULL, n
    assert moe_status(fn, ids=None, scales=None) == NULL           # no logits and no routes
    assert moe_status(fn, ids=None) == NULL and moe_status(fn, gate=GATE, scales=None) == NULL   # half of the routes
    assert moe_status(fn, gate=GATE, logits=None) == NULL and moe_status(fn, logits=FAKE) == NULL
    assert moe_status(fn, shape(world=1, rank=0, copy_experts=2), ori=None) == NULL
    for n in ("x", "w1", "w2", "shared", "ori", "out", "ws"):
        assert moe_status(fn, **{n: FAKE + 8}) == INVALID, n
    for n in ("ids", "scales", "w1s", "w2s"):
        assert moe_status(fn, **{n: FAKE + 2}) == INVALID, n
    assert moe_status(fn, gate=GATE, logits=FAKE + 2) == INVALID and moe_status(fn, gate=GATE, bias=FAKE + 2) == INVALID
    for bad, code in ((dict(groups=5), INVALID), (dict(score=2), INVALID), (dict(dtype=3), INVALID),
                      (dict(scale=float("nan")), INVALID), (dict(groups=16, topk_groups=1), INVALID)):
        assert moe_status(fn, gate={**GATE, **bad}) == code, bad
    assert moe_status(fn, shape(zero_experts=2040), gate=GATE) == UNSUPPORTED
    assert moe_status(fn, bytes_=need - 1) == mdc.MDC_ERR_WORKSPACE
    assert moe_status(fn, shape(bs=0), x=None, out=None, ws=None) == mdc.MDC_OK


# ---- the binding ----

def test_binding_refuses_gmm_int8_tensors():
    z = lambda *s, d=torch.float32: torch.zeros(s).to(d)  # noqa: E731
    i8, i64, bf = torch.int8, torch.int64, torch.bfloat16
    good = dict(a=z(32, 256, d=i8), a_scale=z(32), expert_token_nums=z(2, d=i64), w=z(2, 192, 256, d=i8), w_scale=z(2, 192),
                y=z(32, 192, d=bf))
    for kw, words in [(dict(a=z(32, 256)), "a must be"), (dict(a=z(32, 240, d=i8)), "w has rows"), (dict(a=z(256, d=i8)), "dimensions"),
                      (dict(a_scale=z(31)), "a_scale"), (dict(expert_token_nums=z(1, d=i64)), "expert_token_nums"),
                      (dict(w_scale=z(2, 191)), "w_scale"), (dict(y=z(31, 192, d=bf)), "y holds"), (dict(y=z(32, 192, d=i8)), "y must be"),
                      (dict(a=None), "a must be a tensor"), (dict(w=4096), "w must be a tensor"), (dict(y=None), "y must be a tensor"),
                      (dict(), "on a GPU")]:
        with pytest.raises(ValueError, match=words):
            mdc.mdc_gmm_int8(**{**good, **kw})


def test_binding_refuses_block_norm_tensors():
    bf, f16, f32 = torch.bfloat16, torch.float16, torch.float32
    z = lambda *s, d=bf: torch.zeros(s, dtype=d)  # noqa: E731
    good = dict(x=z(4, 256), weight=z(256), y=z(4, 256))
    for kw, words in [
        (dict(x=None), "x must be a tensor"), (dict(x=z(4, 256, d=f32)), "x must be bf16"), (dict(weight=z(128)), "weight"),
        (dict(weight=z(512)), "weight holds 512"), (dict(weight=z(256, d=f16)), "weight must be"),
        (dict(post_weight=z(256, d=f32)), "post_weight must be"), (dict(post_weight=z(255)), "post_weight"),
        (dict(residual=z(3, 256)), "residual"), (dict(residual=z(4, 256), residual_out=z(4, 256, d=f32)), "residual_out"),
        (dict(gate=z(4, 128)), "gate must have rows"), (dict(gate=z(3, 256)), "gate holds"), (dict(gate=z(4, 256, d=f16)), "gate must be"),
        (dict(gate=z(2, 256), gate_every=1), "gate holds"), (dict(gate=z(2, 256), gate_every=0), "gate_every"),
        (dict(gate=z(4, 1), gate_act="relu"), "gate_act"), (dict(gate=7), "gate must be a tensor"), (dict(y=z(4, 256, d=f32)), "y must be"),
        (dict(q=z(4, 256, d=f32)), "q must be"), (dict(q=z(4, 256, d=torch.int8), q_scale=z(3, d=f32)), "q_scale"),
        (dict(q_scale=z(4, d=f32)), "q_scale without q"), (dict(gate=z(2, 256), gate_every=2), "on a GPU"), (dict(), "on a GPU"),
    ]:
        with pytest.raises(ValueError, match=words):
            mdc.mdc_block_rms_norm(**{**good, **kw})


@pytest.mark.parametrize("int8", [True, False])
def test_binding_refuses_moe_tensors(int8):
    z = lambda *s, d=torch.float32: torch.zeros(s).to(d)  # noqa: E731
    bf, i32, w = torch.bfloat16, torch.int32, torch.int8 if int8 else torch.float8_e4m3fn
    sh = mdc.Shape(1, 0, 4, 256, 2, 3, 0)
    good = dict(x=z(4, 256, d=bf), logits=None, bias=None, expert_ids=z(4, 2, d=i32), expert_scales=z(4, 2),
                w1=z(3, 512, 256, d=w), w1_scale=z(3, 512) if int8 else z(3, 4, 2), w2=z(3, 256, 256, d=w),
                w2_scale=z(3, 256) if int8 else z(3, 2, 2), x_out=z(4, 256, d=bf), workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    call = mdc.mdc_moe if int8 else mdc.mdc_moe_fp8
    for kw, words in [(dict(x=z(4, 256)), "x must be"), (dict(x=z(3, 256, d=bf)), "x holds"), (dict(expert_ids=z(4, 2)), "expert_ids"),
                      (dict(expert_scales=z(4, 1)), "expert_scales"), (dict(w1=z(3, 512, 256, d=bf)), "w1 must be"),
                      (dict(w1_scale=z(1)), "w1_scale"), (dict(w2=z(2, 256, 256, d=w)), "w2 holds"), (dict(w2_scale=z(1)), "w2_scale"),
                      (dict(x_out=z(4, 255, d=bf)), "x_out"), (dict(x_active_mask=z(3, d=torch.uint8)), "x_active_mask"),
                      (dict(shared_expert_x=z(4, 128, d=bf)), "shared_expert_x"), (dict(ori_x=z(4, 256)), "ori_x"),
                      (dict(logits=z(4, 2)), "logits holds"), (dict(logits=z(4, 3, d=torch.float64)), "logits must be"),
                      (dict(logits=z(4, 3), bias=z(2)), "bias"), (dict(logits=z(4, 3), score="tanh"), "score"),
                      (dict(logits=4096), "logits must be a tensor"), (dict(), "on a GPU")]:
        with pytest.raises(ValueError, match=words):
            call(sh, 512, **{**good, **kw})


# ---- the oracles ----

def test_oracle_int8_quant_closed_forms():
    q, s = O.int8_quant(np.array([[0.0, 0, 0], [127, -63.4, 1], [-2, 1, 0.5]]))
    assert s.tolist() == [0, 1, 2 / 127] and q[0].tolist() == [0, 0, 0] and q[1].tolist() == [127, -63, 1]
    assert q[2].tolist() == [-127, 64, 32]   # 63.5 and 31.75


def test_oracle_block_norm_closed_forms():
    x = np.array([[3.0, 4.0], [1.0, 1.0]])
    h, v = O.block_rms_norm(x, np.ones(2), np.array([[2.0], [0.0]]), 1, "none", np.array([[0.0, 0.0], [3.0, 4.0]]), np.ones(2),
                            0.5, 2.0, 0.0, 0.0)
    rms = np.sqrt(12.5)
    assert np.allclose(h, [[3 / rms, 4 / rms], [6, 8]]) and np.allclose(v, [[3 / rms, 4 / rms], [6 / 50 ** 0.5, 8 / 50 ** 0.5]])
    h, v = O.block_rms_norm(x, None, np.array([[0.0, 0.0]]), 2, "sigmoid", None, None, 1, 1, 0, 0)
    assert np.allclose(h, x / 2) and v is None


def test_oracle_moe_routes_closed_forms():
    ids = np.array([[0, 5], [4, 4], [6, 9], [-1, 2]])
    sc = np.array([[1.0, 2], [3, 4], [5, 6], [7, 8]])
    w, has, cp, present, dropped = O.moe_routes(ids, sc, None, 4, 2, 6, 1, 2)   # routed 0..5, here 4 and 5; zero 6; copy 7, 8
    assert w.tolist() == [[0, 2], [7, 0], [0, 0], [0, 0]] and has.tolist() == [[False, True], [True, False]] + [[False] * 2] * 2
    assert cp.tolist() == [0, 0, 0, 0] and present.tolist() == [3, 7, 5, 8] and dropped == 2
    _, _, cp, present, dropped = O.moe_routes(np.array([[7, 8]]), np.array([[1.0, 2]]), np.array([[1, 0]]), 4, 2, 6, 1, 2)
    assert cp.tolist() == [1] and present.tolist() == [1] and dropped == 0
