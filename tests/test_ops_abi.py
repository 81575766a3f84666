"""Argument checks of the gate, the norm and the fp8 products (no GPU needed:
every call returns before anything is enqueued), and properties of the 64-bit
oracle that the GPU tests use."""
import ctypes

import numpy as np
import pytest
import torch

import combine_route_histogram_amd as mdc
from oracle import ops64 as O

FAKE = 1 << 20
P = ctypes.c_void_p


def gate_status(shape=None, logits=FAKE, bias=None, ids=FAKE, scales=FAKE, params=True, **over):
    sh = shape or mdc.Shape(2, 0, 16, 64, 4, 32, 0)
    kw = dict(dtype=mdc.MDC_DTYPE_FP32, score=mdc.MDC_GATE_SOFTMAX, groups=1, topk_groups=1, group_top=1,
              renormalise=1, scale=1.0)
    kw.update(over)
    return mdc._lib.mdc_gate(sh.c(), mdc.mdc_gate_params(**kw) if params else None, P(logits), P(bias), P(ids),
                             P(scales), None)


@pytest.mark.parametrize("kw,want", [
    (dict(params=False), mdc.MDC_ERR_NULLPTR), (dict(logits=None), mdc.MDC_ERR_NULLPTR),
    (dict(ids=None), mdc.MDC_ERR_NULLPTR), (dict(scales=None), mdc.MDC_ERR_NULLPTR),
    (dict(dtype=3), mdc.MDC_ERR_INVALID), (dict(dtype=-1), mdc.MDC_ERR_INVALID), (dict(score=2), mdc.MDC_ERR_INVALID),
    (dict(groups=0), mdc.MDC_ERR_INVALID), (dict(groups=5), mdc.MDC_ERR_INVALID),
    (dict(groups=8, topk_groups=0), mdc.MDC_ERR_INVALID), (dict(groups=8, topk_groups=9), mdc.MDC_ERR_INVALID),
    (dict(groups=8, topk_groups=2, group_top=3), mdc.MDC_ERR_INVALID),
    (dict(groups=8, topk_groups=2, group_top=0), mdc.MDC_ERR_INVALID),
    (dict(groups=32, topk_groups=8, group_top=2), mdc.MDC_ERR_INVALID),   # groups of one id
    (dict(groups=16, topk_groups=1), mdc.MDC_ERR_INVALID),                # 2 open ids, K = 4
    (dict(renormalise=2), mdc.MDC_ERR_INVALID), (dict(scale=float("inf")), mdc.MDC_ERR_INVALID),
    (dict(scale=float("nan")), mdc.MDC_ERR_INVALID), (dict(logits=FAKE + 2), mdc.MDC_ERR_INVALID),
    (dict(dtype=mdc.MDC_DTYPE_BF16, logits=FAKE + 1), mdc.MDC_ERR_INVALID), (dict(ids=FAKE + 2), mdc.MDC_ERR_INVALID),
    (dict(bias=FAKE + 1), mdc.MDC_ERR_INVALID),
    (dict(shape=mdc.Shape(1, 0, 16, 64, 4, 2040, 0, zero_experts=8, copy_experts=8)), mdc.MDC_ERR_UNSUPPORTED),
    (dict(shape=mdc.Shape(1, 0, 16, 64, 1, 256, 0), groups=128, topk_groups=128), mdc.MDC_ERR_UNSUPPORTED),
    (dict(shape=mdc.Shape(1, 0, 16, 64, 17, 32, 0)), mdc.MDC_ERR_UNSUPPORTED),
    (dict(shape=mdc.Shape(1, 0, -1, 64, 2, 32, 0)), mdc.MDC_ERR_INVALID),
    (dict(shape=mdc.Shape(1, 0, 0, 64, 2, 32, 0), logits=None), mdc.MDC_OK),   # no tokens
])
def test_gate_argument_checks(kw, want):
    assert gate_status(**kw) == want


def norm_status(x=FAKE, res=None, w=FAKE, res_out=None, y=FAKE, q=None, s=None, params=True, **over):
    kw = dict(rows=4, hidden=64, dtype=mdc.MDC_DTYPE_BF16, residual_dtype=mdc.MDC_DTYPE_BF16,
              weight_dtype=mdc.MDC_DTYPE_BF16, quant=mdc.MDC_QUANT_NONE, eps=1e-6)
    kw.update(over)
    return mdc._lib.mdc_add_rms_norm(mdc.mdc_norm_params(**kw) if params else None, P(x), P(res), P(w), P(res_out),
                                     P(y), P(q), P(s), None)


@pytest.mark.parametrize("kw,want", [
    (dict(params=False), mdc.MDC_ERR_NULLPTR), (dict(x=None), mdc.MDC_ERR_NULLPTR), (dict(w=None), mdc.MDC_ERR_NULLPTR),
    (dict(y=None), mdc.MDC_ERR_NULLPTR),   # no output at all
    (dict(quant=mdc.MDC_QUANT_INT8), mdc.MDC_ERR_NULLPTR), (dict(quant=mdc.MDC_QUANT_FP8, q=FAKE), mdc.MDC_ERR_NULLPTR),
    (dict(q=FAKE, s=FAKE), mdc.MDC_ERR_NULLPTR),   # q without a quant mode
    (dict(s=FAKE), mdc.MDC_ERR_NULLPTR),
    (dict(dtype=mdc.MDC_DTYPE_FP32), mdc.MDC_ERR_INVALID),
    (dict(residual_dtype=mdc.MDC_DTYPE_FP16), mdc.MDC_ERR_INVALID),
    (dict(weight_dtype=mdc.MDC_DTYPE_FP16), mdc.MDC_ERR_INVALID), (dict(quant=3), mdc.MDC_ERR_INVALID),
    (dict(rows=-1), mdc.MDC_ERR_INVALID), (dict(hidden=0), mdc.MDC_ERR_INVALID), (dict(hidden=60), mdc.MDC_ERR_INVALID),
    (dict(eps=-1.0), mdc.MDC_ERR_INVALID), (dict(eps=float("nan")), mdc.MDC_ERR_INVALID),
    (dict(eps=float("inf")), mdc.MDC_ERR_INVALID), (dict(x=FAKE + 8), mdc.MDC_ERR_INVALID),
    (dict(w=FAKE + 8), mdc.MDC_ERR_INVALID), (dict(res=FAKE + 8), mdc.MDC_ERR_INVALID),
    (dict(res_out=FAKE + 8), mdc.MDC_ERR_INVALID), (dict(y=FAKE + 8), mdc.MDC_ERR_INVALID),
    (dict(quant=mdc.MDC_QUANT_FP8, q=FAKE + 4, s=FAKE), mdc.MDC_ERR_INVALID),
    (dict(quant=mdc.MDC_QUANT_FP8, q=FAKE, s=FAKE + 2), mdc.MDC_ERR_INVALID),
    (dict(hidden=32776), mdc.MDC_ERR_UNSUPPORTED), (dict(rows=2 ** 31), mdc.MDC_ERR_UNSUPPORTED),
    (dict(rows=0, x=None, w=None, y=None), mdc.MDC_OK),
])
def test_norm_argument_checks(kw, want):
    assert norm_status(**kw) == want


def gmm_status(A=64, L=4, n=64, k=128, a=FAKE, sa=FAKE, nums=FAKE, w=FAKE, sw=FAKE, y=FAKE):
    return mdc._lib.mdc_gmm_fp8(A, L, n, k, P(a), P(sa), P(nums), P(w), P(sw), P(y), None)


@pytest.mark.parametrize("kw,want", [
    (dict(a=None), mdc.MDC_ERR_NULLPTR), (dict(sa=None), mdc.MDC_ERR_NULLPTR), (dict(nums=None), mdc.MDC_ERR_NULLPTR),
    (dict(w=None), mdc.MDC_ERR_NULLPTR), (dict(sw=None), mdc.MDC_ERR_NULLPTR), (dict(y=None), mdc.MDC_ERR_NULLPTR),
    (dict(A=-1), mdc.MDC_ERR_INVALID), (dict(L=0), mdc.MDC_ERR_INVALID), (dict(n=0), mdc.MDC_ERR_INVALID),
    (dict(n=60), mdc.MDC_ERR_INVALID), (dict(k=0), mdc.MDC_ERR_INVALID), (dict(k=136), mdc.MDC_ERR_INVALID),
    (dict(a=FAKE + 8), mdc.MDC_ERR_INVALID), (dict(w=FAKE + 8), mdc.MDC_ERR_INVALID),
    (dict(y=FAKE + 8), mdc.MDC_ERR_INVALID), (dict(sa=FAKE + 2), mdc.MDC_ERR_INVALID),
    (dict(nums=FAKE + 4), mdc.MDC_ERR_INVALID),
    (dict(L=2049), mdc.MDC_ERR_UNSUPPORTED), (dict(A=2 ** 31), mdc.MDC_ERR_UNSUPPORTED),
    (dict(n=1 << 16, k=1 << 15), mdc.MDC_ERR_UNSUPPORTED), (dict(n=8, k=(1 << 22) + 16), mdc.MDC_ERR_UNSUPPORTED),
    (dict(A=2 ** 31 - 1, n=1 << 14, k=16), mdc.MDC_ERR_UNSUPPORTED),
    (dict(A=0, a=None, w=None, y=None), mdc.MDC_OK),
])
def test_gmm_argument_checks(kw, want):
    assert gmm_status(**kw) == want


FFN = mdc.Shape(world=8, rank=0, bs=32, hidden=512, topk=8, num_experts=64, capacity=2048)


@pytest.mark.parametrize("quant_input", [False, True])
def test_ffn_fp8_argument_checks(quant_input):
    need = mdc.mdc_ffn_fp8_workspace(FFN, 512)
    # status block, q1 + s1, q2 + s2 at least
    assert need >= mdc.MDC_STATUS_BYTES + 2048 * (512 + 4 * 4) + 2048 * (256 + 2 * 4)
    for shape, inter, code in ((FFN, 0, mdc.MDC_ERR_INVALID), (FFN, 384, mdc.MDC_ERR_UNSUPPORTED),
                               (mdc.Shape(8, 0, 32, 520, 8, 64, 2048), 512, mdc.MDC_ERR_UNSUPPORTED),
                               (mdc.Shape(8, 0, 32, 512, 8, 60, 2048), 512, mdc.MDC_ERR_INVALID),
                               (mdc.Shape(8, 0, 32, 1 << 20, 8, 64, 2048), 1 << 12, mdc.MDC_ERR_UNSUPPORTED)):
        with pytest.raises(mdc.MdcError) as ei:
            mdc.mdc_ffn_fp8_workspace(shape, inter)
        assert ei.value.status == code
    names = ["x", "s", "nums", "w1", "w1s", "w2", "w2s", "y", "ws"]

    def call(bytes_=need, shape=FFN, **over):
        v = [over.get(n, FAKE) for n in names]
        head = v[:2] if quant_input else v[:1]
        fn = mdc._lib.mdc_ffn_fp8_quant_input if quant_input else mdc._lib.mdc_ffn_fp8
        return fn(shape.c(), 512, *[P(a) for a in head + v[2:]], bytes_, None)

    for n in names:
        if n != "s" or quant_input:
            assert call(**{n: None}) == mdc.MDC_ERR_NULLPTR, n
    for n in ("x", "w1", "w2", "y", "ws"):
        assert call(**{n: FAKE + 8}) == mdc.MDC_ERR_INVALID, n
    assert call(bytes_=need - 1) == mdc.MDC_ERR_WORKSPACE
    assert call(shape=mdc.Shape(8, 0, 32, 512, 8, 64, 0), x=None, y=None) == mdc.MDC_OK


# ---- the binding ----

def _gate_tensors(**over):
    a = dict(logits=torch.zeros((2, 8, 32)), bias=torch.zeros(32), expert_ids=torch.zeros((2, 8, 2), dtype=torch.int32),
             expert_scales=torch.zeros((2, 8, 2)))
    a.update(over)
    return a


@pytest.mark.parametrize("over,words", [
    (dict(logits=torch.zeros((2, 8, 31))), "logits"), (dict(logits=torch.zeros((2, 8, 32), dtype=torch.float64)), "logits"),
    (dict(bias=torch.zeros(31)), "bias"), (dict(bias=torch.zeros(32, dtype=torch.bfloat16)), "bias"),
    (dict(expert_ids=torch.zeros((2, 8, 2), dtype=torch.int64)), "expert_ids"),
    (dict(expert_scales=torch.zeros((2, 8, 1))), "expert_scales"), (dict(score="tanh"), "score"),
    (dict(), "on a GPU"),
])
def test_binding_refuses_gate_tensors(over, words):
    with pytest.raises(ValueError, match=words):
        mdc.mdc_gate(mdc.Shape(2, 0, 8, 64, 2, 32, 0), **_gate_tensors(**over))


def test_binding_refuses_norm_tensors():
    bf, f16, f32 = torch.bfloat16, torch.float16, torch.float32
    x, w = torch.zeros((4, 256), dtype=bf), torch.zeros(256, dtype=bf)
    z = lambda *s, d=bf: torch.zeros(s, dtype=d)  # noqa: E731
    for kw, words in [
        (dict(x=z(4, 256, d=f32)), "x must be"), (dict(weight=z(128)), "weight holds"),
        (dict(weight=z(256, d=f16)), "weight"), (dict(residual=z(4, 256, d=f16)), "residual"),
        (dict(residual=z(3, 256)), "residual"), (dict(residual=z(4, 256), residual_out=z(4, 256, d=f32)), "residual_out"),
        (dict(y=z(4, 256, d=f32)), "y must be"), (dict(y=z(4, 128)), "y holds"), (dict(q=z(4, 256, d=f32)), "q must be"),
        (dict(q=z(4, 256, d=torch.int8), q_scale=z(3, d=f32)), "q_scale"),
        (dict(q=z(4, 256, d=torch.float8_e4m3fn), q_scale=z(7, d=f32)), "q_scale"),
        (dict(q_scale=z(4, d=f32)), "q_scale without q"), (dict(y=z(4, 256)), "on a GPU"),
    ]:
        a = dict(x=x, weight=w)
        a.update(kw)
        with pytest.raises(ValueError, match=words):
            mdc.mdc_add_rms_norm(**a)


def test_binding_refuses_product_tensors():
    f8, f32, i64 = torch.float8_e4m3fn, torch.float32, torch.int64
    z = lambda *s, d=f32: torch.zeros(s).to(d)  # noqa: E731
    good = dict(a=z(32, 256, d=f8), a_scale=z(32, 2), expert_token_nums=z(2, d=i64), w=z(2, 192, 256, d=f8),
                w_scale=z(2, 2, 2), y=z(32, 192, d=torch.bfloat16))
    for kw, words in [
        (dict(a=z(32, 256)), "a must be"), (dict(a=z(32, 240, d=f8)), "w has rows"), (dict(a=z(256, d=f8)), "dimensions"),
        (dict(a_scale=z(31, 2)), "a_scale"), (dict(expert_token_nums=z(1, d=i64)), "expert_token_nums"),
        (dict(w_scale=z(2, 1, 2)), "w_scale"), (dict(y=z(31, 192, d=torch.bfloat16)), "y holds"),
        (dict(y=z(32, 192)), "y must be"), (dict(), "on a GPU"),
        (dict(a=z(256, 32, d=f8).t()), "contiguous|on a GPU"),
    ]:
        with pytest.raises(ValueError, match=words):
            mdc.mdc_gmm_fp8(**{**good, **kw})
    sh = mdc.Shape(1, 0, 32, 256, 1, 2, 32)
    ffn = dict(expand_x=z(32, 256, d=torch.bfloat16), expert_token_nums=z(2, d=i64), w1=z(2, 512, 256, d=f8),
               w1_scale=z(2, 4, 2), w2=z(2, 256, 256, d=f8), w2_scale=z(2, 2, 2), y=z(32, 256, d=torch.bfloat16),
               workspace=torch.zeros(16, dtype=torch.uint8))
    for kw, words in [(dict(expand_x=z(31, 256, d=torch.bfloat16)), "expand_x"), (dict(w1_scale=z(2, 4, 1)), "w1_scale"),
                      (dict(w1=z(2, 256, 256, d=f8)), "w1"), (dict(w2=z(2, 256, 128, d=f8)), "w2"),
                      (dict(w2_scale=z(2, 1, 2)), "w2_scale"), (dict(y=z(31, 256, d=torch.bfloat16)), "y"),
                      (dict(), "on a GPU")]:
        with pytest.raises(ValueError, match=words):
            mdc.mdc_ffn_fp8(sh, 512, **{**ffn, **kw})


# ---- the oracle ----

def test_oracle_e4m3_rounds_as_the_nearest_code():
    values = O.e4m3_values()
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(values, codes, equal_nan=True)
    v = np.sort(values[np.isfinite(values)])
    v = np.unique(v)
    assert np.array_equal(O.e4m3_round(v), v)
    mid = (v[1:] + v[:-1]) / 2                      # halves go to the even code, everything else to the nearest
    lo, hi = O.e4m3_round(mid - 1e-12 * np.abs(mid) - 1e-15), O.e4m3_round(mid + 1e-12 * np.abs(mid) + 1e-15)
    assert np.array_equal(lo, v[:-1]) and np.array_equal(hi, v[1:])
    t = torch.from_numpy(mid).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.e4m3_round(mid), t)


def test_oracle_gate_closed_forms():
    ids, w = O.gate([[0.0, 1.0, 1.0, -np.inf], [np.nan, -np.inf, 5.0, -np.inf]], None, 3, renormalise=True)
    assert ids.tolist() == [[1, 2, 0], [2, -1, -1]]
    assert np.allclose(w[0], np.exp([0, 0, -1]) / np.exp([0, 0, -1]).sum()) and w[1].tolist() == [1, 0, 0]
    ids, _ = O.gate([[3.0, 0.0, 2.0, 1.9]], np.zeros(4), 2, "sigmoid", groups=2, topk_groups=1, group_top=2)
    assert ids.tolist() == [[2, 3]]   # 0.95 + 0.5 < 0.88 + 0.87
