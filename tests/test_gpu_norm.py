"""mdc_add_rms_norm against the 64-bit oracle."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_route_histogram_amd as mdc  # noqa: E402
from oracle import ops64 as O  # noqa: E402

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
# fp32 arithmetic of v: the sum of squares takes at most 64 additions per lane and wave, then the mean, the root, the
# quotient and two products
V_REL = 80 * 2.0 ** -24


def make(rows, H, dtype, res_dtype, w_dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, H), generator=g).to(dtype)
    res = None if res_dtype is None else (3 * torch.randn((rows, H), generator=g) *
                                          torch.exp(torch.randn((H,), generator=g))).to(res_dtype)
    return x, res, (1 + 0.3 * torch.randn((H,), generator=g)).to(w_dtype)


def np64(t):
    return None if t is None else t.double().cpu().numpy()


def half_step(t):
    return torch.finfo(t).eps / 2


def check_rounded(got, want, rel, dtype):
    """A value rounded once to dtype from one that is off by rel (subnormals: half their step)."""
    tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    err = np.abs(np64(got) - want)
    assert np.all(err <= (half_step(dtype) + 1.01 * rel) * np.abs(want) + tiny), (err / (np.abs(want) + 1e-30)).max()


def check_q(q, s, v, quant):
    s = np64(s)
    if quant == "int8":
        amax = np.abs(v).max(1)
        assert np.all(np.abs(s - amax / 127) <= (V_REL + 2.0 ** -22) * amax / 127)
        # half a code, and the fp32 error of v and of the quotient
        assert np.all(np.abs(np64(q) * s[:, None] - v) <= s[:, None] * (0.5 + 127 * (V_REL + 2.0 ** -22)))
        assert np.all(np.abs(np64(q)) <= 127)
        return
    H = v.shape[1]
    for b in range(-(-H // 128)):
        part = v[:, b * 128:(b + 1) * 128]
        amax = np.abs(part).max(1)
        want = np.where(amax > 0, np.maximum(amax, O.AMAX_MIN), 0) / 448
        assert np.all(np.abs(s[:, b] - want) <= (V_REL + 2.0 ** -22) * want)
        got = np64(q[:, b * 128:(b + 1) * 128].float()) * s[:, b:b + 1]
        # half an e4m3 step: 2^-4 of the value, 2^-10 of the scale below 2^-6 of it
        assert np.all(np.abs(got - part) <= (2.0 ** -4 + 2 * V_REL) * np.abs(part) + 2.0 ** -10 * s[:, b:b + 1])


def run_and_check(rows, H, dtype, res_dtype, w_dtype, quant, with_y, with_res_out=True, seed=0, tensors=None, eps=1e-6):
    x, res, w = tensors if tensors is not None else make(rows, H, dtype, res_dtype, w_dtype, seed)
    guard = 2   # rows behind the last one stay as they were
    dev = lambda *s, d: torch.full(s, 7, device=DEV).to(d)  # noqa: E731
    y = dev(rows + guard, H, d=dtype) if with_y else None
    out_t = res_dtype if res_dtype is not None else dtype
    rout = dev(rows + guard, H, d=out_t) if with_res_out else None
    q = s = None
    if quant != "none":
        q = dev(rows + guard, H, d=torch.int8 if quant == "int8" else E4M3)
        s = dev(rows + guard, 1 if quant == "int8" else -(-H // 128), d=torch.float32)
    mdc.mdc_add_rms_norm(x.to(DEV), w.to(DEV), residual=None if res is None else res.to(DEV), residual_out=rout, y=y,
                         q=q, q_scale=s, eps=eps)
    torch.cuda.synchronize()
    for t in (y, rout, q, s):
        assert t is None or (t[rows:].float() == 7).all()
    h, v = O.add_rms_norm(np64(x), np64(res), np64(w), eps)
    if with_res_out:
        check_rounded(rout[:rows], h, 2.0 ** -24, out_t)
    if with_y:
        check_rounded(y[:rows], v, V_REL, dtype)
    if quant != "none":
        check_q(q[:rows].cpu(), s[:rows].reshape(rows, -1)[:, 0] if quant == "int8" else s[:rows], v, quant)


BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("quant", ["none", "int8", "fp8"])
@pytest.mark.parametrize("rows,H", [(1, 8), (1, 7168), (3, 128), (5, 136), (2, 504), (7, 512), (3, 520), (33, 1000),
                                    (4, 5000), (9, 7168), (3, 8192), (2, 8200), (2, 16384), (1, 32768), (300, 256)])
def test_norm_sizes(rows, H, quant):
    run_and_check(rows, H, BF, BF, BF, quant, with_y=True, seed=H)


@pytest.mark.parametrize("quant", ["none", "int8", "fp8"])
@pytest.mark.parametrize("dtype,res,w", [(BF, F32, BF), (BF, BF, F32), (BF, F32, F32), (BF, None, BF), (F16, F16, F16),
                                         (F16, F32, F16), (F16, F16, F32), (F16, F32, F32), (F16, None, F32)])
def test_norm_types(dtype, res, w, quant):
    run_and_check(6, 1160, dtype, res, w, quant, with_y=quant != "fp8", seed=3)


@pytest.mark.parametrize("quant", ["int8", "fp8"])
def test_norm_single_outputs(quant):
    run_and_check(5, 640, BF, BF, BF, quant, with_y=False, with_res_out=False, seed=4)
    run_and_check(5, 640, BF, BF, BF, "none", with_y=False, with_res_out=True, seed=5)
    run_and_check(5, 640, BF, None, BF, "none", with_y=True, with_res_out=False, seed=6)


@pytest.mark.parametrize("quant", ["int8", "fp8"])
def test_norm_zeros_and_extreme_rows(quant):
    """Zero rows and runs, a run far below the others, rows near the ends of the range."""
    x, res, w = make(6, 512, BF, BF, F32, 8)
    x[0], res[0] = 0, 0
    x[1, 128:256], res[1, 128:256] = 0, 0
    x[2], res[2] = x[2] * 1e-12, 0
    x[3, 256:384], res[3, 256:384] = x[3, 256:384] * 1e-30, 0
    x[4], res[4] = x[4] * 1e17, 0
    w[5] = 0
    run_and_check(6, 512, BF, BF, F32, quant, True, tensors=(x, res, w))
    x, s = torch.zeros((2, 256), dtype=BF, device=DEV), torch.ones((2, 2 if quant == "fp8" else 1), device=DEV)
    q = torch.ones((2, 256), device=DEV).to(E4M3 if quant == "fp8" else torch.int8)
    mdc.mdc_add_rms_norm(x, torch.ones(256, dtype=BF, device=DEV), q=q, q_scale=s)
    assert (q.float() == 0).all() and (s == 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("quant", ["int8", "fp8"])
def test_norm_non_finite_rows_stay_visible(bad, quant):
    """A NaN or infinity in a row shows in that row's scales, and in no other row."""
    x, res, w = make(4, 512, BF, BF, BF, 9)
    x[2, 300] = bad
    y = torch.empty((4, 512), dtype=BF, device=DEV)
    q = torch.empty((4, 512), device=DEV).to(E4M3 if quant == "fp8" else torch.int8)
    s = torch.empty((4, 4 if quant == "fp8" else 1), device=DEV)
    mdc.mdc_add_rms_norm(x.to(DEV), w.to(DEV), residual=res.to(DEV), y=y, q=q, q_scale=s)
    assert not torch.isfinite(s[2]).all() and torch.isfinite(s[[0, 1, 3]]).all()
    assert torch.isfinite(y[[0, 1, 3]]).all()


@pytest.mark.parametrize("H", [512, 7168, 16384])
def test_norm_in_place(H):
    """residual_out may be residual or x itself, y may be x itself."""
    x, res, w = (t.to(DEV) for t in make(5, H, BF, BF, BF, 10))
    want_r, want_y = torch.empty_like(x), torch.empty_like(x)
    mdc.mdc_add_rms_norm(x, w, residual=res, residual_out=want_r, y=want_y)
    r2, x2 = res.clone(), x.clone()
    mdc.mdc_add_rms_norm(x2, w, residual=r2, residual_out=r2, y=x2)
    assert torch.equal(r2, want_r) and torch.equal(x2, want_y)
    x3, y3 = x.clone(), torch.empty_like(x)
    mdc.mdc_add_rms_norm(x3, w, residual=res, residual_out=x3, y=y3)
    assert torch.equal(x3, want_r) and torch.equal(y3, want_y)


def test_norm_on_another_stream_and_in_a_graph():
    x, res, w = (t.to(DEV) for t in make(40, 1024, BF, F32, BF, 12))
    out = lambda: dict(residual_out=torch.empty_like(res), y=torch.empty_like(x),  # noqa: E731
                       q=torch.empty((40, 1024), device=DEV).to(E4M3), q_scale=torch.empty((40, 8), device=DEV))
    a, b = out(), out()
    call = mdc.prepare_add_rms_norm(x, w, residual=res, **a)
    call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mdc.mdc_add_rms_norm(x, w, residual=res, **b)
    torch.cuda.synchronize()
    for k in a:
        assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mdc.mdc_add_rms_norm(x, w, residual=res, **b)
    for rep in range(3):
        x.copy_(torch.randn((40, 1024), device=DEV))
        b["y"].zero_()
        graph.replay()
        call()
        torch.cuda.synchronize()
        for k in a:
            assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), (rep, k)
