"""mdc_block_rms_norm against the 64-bit oracle."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_route_histogram_amd as mdc  # noqa: E402
from oracle import ops64 as O  # noqa: E402
from tests.test_gpu_norm import check_q, np64  # noqa: E402

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32

# fp32 errors, relative: a mean of squares takes at most 64 additions of positive terms per lane and wave, then the mean, the
# root and the quotient (80 roundings, halved by the root).  The block's term of h: that factor, the products with post_weight,
# act(gate) and block_scale (the activation within 8 steps), the FMA.  Then v adds the second norm on top of h's error.
U_REL = 56 * 2.0 ** -24
V_REL = 56 * 2.0 ** -24


def make(rows, H, dtype, res, w, gate, every, gate_dtype, post, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    t = dict(x=(2 * n(rows, H)).to(dtype), weight=(1 + 0.3 * n(H)).to(w))
    if post:
        t["post_weight"] = (1 + 0.3 * n(H)).to(w)
    if res is not None:
        t["residual"] = (3 * n(rows, H) * torch.exp(n(H))).to(res)
    if gate is not None:
        t["gate"] = (0.5 + n(-(-rows // every), H if gate == "wide" else 1)).to(gate_dtype)
    return t


def run_and_check(t, every=1, act="none", quant="fp8", with_y=True, with_res_out=True, block_scale=0.75,
                  residual_scale=1.25, post_eps=1e-5, eps=1e-6, weighted=True):
    x, res = t["x"], t.get("residual")
    rows, H = x.shape
    dtype, out_t = x.dtype, x.dtype if res is None else res.dtype
    dev = lambda *s, d: torch.full(s, 7, device=DEV).to(d)  # noqa: E731
    guard = 2   # rows behind the last one stay as they were
    out = dict(residual_out=dev(rows + guard, H, d=out_t) if with_res_out else None,
               y=dev(rows + guard, H, d=dtype) if with_y else None, q=None, q_scale=None)
    if quant != "none":
        out["q"] = dev(rows + guard, H, d=torch.int8 if quant == "int8" else E4M3)
        out["q_scale"] = dev(rows + guard, 1 if quant == "int8" else -(-H // 128), d=F32)
    args = {k: v.to(DEV) for k, v in t.items()}
    if not weighted:
        args.pop("weight")
    mdc.mdc_block_rms_norm(**args, **out, gate_every=every, gate_act=act, block_scale=block_scale,
                           residual_scale=residual_scale, post_eps=post_eps, eps=eps)
    torch.cuda.synchronize()
    for o in out.values():
        assert o is None or (o[rows:].float() == 7).all()
    n64 = {k: np64(v) for k, v in t.items()}
    full = (n64["x"], n64.get("post_weight"), n64.get("gate"), every, act, n64.get("residual"),
            n64["weight"] if weighted else None, block_scale, residual_scale, post_eps, eps)
    h, v = O.block_rms_norm(*full)
    # the two terms of h may cancel: its error is that of their sizes
    term = np.abs(h - residual_scale * n64["residual"]) if res is not None else np.abs(h)
    size = term + (np.abs(residual_scale * n64["residual"]) if res is not None else 0)
    h_err = U_REL * size
    if with_res_out:
        eps_t = torch.finfo(out_t).eps / 2
        tiny = torch.finfo(out_t).smallest_normal * torch.finfo(out_t).eps
        err = np.abs(np64(out["residual_out"][:rows]) - h)
        assert np.all(err <= eps_t * np.abs(h) + 1.01 * h_err + tiny), (err / (np.abs(h) + 1e-30)).max()
    if not weighted:
        return
    # v: h's error by element and, through the row's norm, at most the error of the whole row
    inv = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    row = np.sqrt((h_err ** 2).mean(1, keepdims=True)) * inv
    v_err = np.abs(inv * n64["weight"]) * h_err + (row + V_REL) * np.abs(v)
    if with_y:
        eps_t = torch.finfo(dtype).eps / 2
        tiny = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
        err = np.abs(np64(out["y"][:rows]) - v)
        assert np.all(err <= eps_t * np.abs(v) + 1.01 * v_err + tiny), (err / (np.abs(v) + 1e-30)).max()
    if quant == "none":
        return
    s, q = np64(out["q_scale"][:rows]), out["q"][:rows].cpu()
    if quant == "int8":
        amax = np.abs(v).max(1)
        off = v_err.max(1) + 2.0 ** -21 * amax
        assert np.all(np.abs(s[:, 0] - amax / 127) <= off / 127)
        assert np.all(np.abs(np64(q) * s - v) <= s * 0.5 + v_err + off[:, None])
        return
    for b in range(-(-H // 128)):
        part, pe = v[:, b * 128:(b + 1) * 128], v_err[:, b * 128:(b + 1) * 128]
        amax = np.abs(part).max(1)
        want = np.where(amax > 0, np.maximum(amax, O.AMAX_MIN), 0) / 448
        off = pe.max(1) + 2.0 ** -21 * amax
        assert np.all(np.abs(s[:, b] - want) <= off / 448)
        got = np64(q[:, b * 128:(b + 1) * 128].float()) * s[:, b:b + 1]
        # half an e4m3 step: 2^-4 of the value, 2^-10 of the scale below 2^-6 of it
        tol = 2.0 ** -4 * np.abs(part) + 2.0 ** -10 * s[:, b:b + 1] + 1.07 * pe + off[:, None]
        assert np.all(np.abs(got - part) <= tol)


@pytest.mark.parametrize("quant", ["none", "int8", "fp8"])
@pytest.mark.parametrize("rows,H", [(1, 8), (1, 7168), (3, 128), (5, 136), (2, 504), (7, 512), (3, 520), (33, 1000),
                                    (4, 5000), (9, 7168), (3, 8192), (2, 8200), (2, 16384), (1, 32768), (300, 256)])
def test_sizes(rows, H, quant):
    run_and_check(make(rows, H, BF, BF, BF, "wide", 1, BF, True, H), quant=quant)


@pytest.mark.parametrize("quant", ["none", "int8", "fp8"])
@pytest.mark.parametrize("dtype,res,w,gate", [(BF, F32, BF, F32), (BF, BF, F32, BF), (BF, F32, F32, F32), (BF, None, BF, BF),
                                              (F16, F16, F16, F16), (F16, F32, F16, F32), (F16, F16, F32, F16),
                                              (F16, F32, F32, F16), (F16, None, F32, F32)])
def test_types(dtype, res, w, gate, quant):
    run_and_check(make(6, 1160, dtype, res, w, "wide", 2, gate, True, 3), every=2, quant=quant, with_y=quant != "fp8")


@pytest.mark.parametrize("act", ["none", "sigmoid", "tanh"])
@pytest.mark.parametrize("gate,every", [(None, 1), ("wide", 1), ("wide", 7), ("wide", 3), ("one", 1), ("one", 5),
                                        ("one", 7), ("wide", 1000)])
@pytest.mark.parametrize("post", [True, False])
def test_gates(gate, every, act, post):
    for gate_dtype in (BF, F32):
        run_and_check(make(7, 640, BF, BF, BF, gate, every, gate_dtype, post, every), every=every, act=act)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("res", [None, BF, F32])
def test_parts_left_out(post, res):
    t = make(5, 640, BF, res, BF, None, 1, BF, post, 4)
    run_and_check(t, quant="none", with_res_out=False)
    run_and_check(t, quant="none", with_y=False)
    run_and_check(t, quant="none", with_y=False, weighted=False)
    run_and_check(t, quant="int8", with_y=False, with_res_out=False)
    run_and_check(t, block_scale=0.0 if res is not None else -1.0, residual_scale=-2.0)
    if res is not None:
        run_and_check(t, residual_scale=0.0)


def test_saturated_gates():
    """Gates at the ends of the range: sigmoid and tanh go to 0, 1 and -1, never to NaN."""
    t = make(4, 256, BF, F32, BF, "wide", 1, F32, True, 5)
    t["gate"][0] = 200.0
    t["gate"][1] = -80.0
    t["gate"][2] = 3e38
    for act in ("sigmoid", "tanh"):
        run_and_check(t, act=act)
    t["gate"][3] = -3e38
    out = torch.empty((4, 256), device=DEV)
    mdc.mdc_block_rms_norm(**{k: v.to(DEV) for k, v in t.items()}, residual_out=out, gate_act="sigmoid")
    assert torch.equal(out[3].cpu(), t["residual"][3])   # the block is shut


def test_zero_rows():
    t = make(4, 512, BF, BF, BF, "one", 1, BF, True, 6)
    t["x"][0], t["residual"][0] = 0, 0
    t["gate"][1] = 0
    t["residual"][2] = 0
    for quant in ("fp8", "int8"):
        run_and_check(t, quant=quant)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["x", "residual", "gate"])
def test_non_finite_rows_stay_visible(bad, where):
    """A NaN or infinity shows in its row's outputs, and in no other row."""
    t = make(4, 512, BF, BF, BF, "wide", 1, BF, True, 9)
    t[where][2, 300] = bad
    y, q = torch.empty((4, 512), dtype=BF, device=DEV), torch.empty((4, 512), device=DEV).to(E4M3)
    s, r = torch.empty((4, 4), device=DEV), torch.empty((4, 512), dtype=BF, device=DEV)
    mdc.mdc_block_rms_norm(**{k: v.to(DEV) for k, v in t.items()}, residual_out=r, y=y, q=q, q_scale=s)
    assert not torch.isfinite(s[2]).all() and not torch.isfinite(r[2]).all()
    for o in (s, r, y, q.float()):
        assert torch.isfinite(o[[0, 1, 3]]).all()


@pytest.mark.parametrize("H", [512, 7168, 16384])
def test_in_place(H):
    """residual_out may be residual or x itself, y may be x itself."""
    t = {k: v.to(DEV) for k, v in make(5, H, BF, BF, BF, "wide", 1, BF, True, 10).items()}
    want_r, want_y = torch.empty_like(t["x"]), torch.empty_like(t["x"])
    mdc.mdc_block_rms_norm(**t, residual_out=want_r, y=want_y)
    r2, x2 = t["residual"].clone(), t["x"].clone()
    mdc.mdc_block_rms_norm(**{**t, "x": x2, "residual": r2}, residual_out=r2, y=x2)
    assert torch.equal(r2, want_r) and torch.equal(x2, want_y)
    x3, y3 = t["x"].clone(), torch.empty_like(t["x"])
    mdc.mdc_block_rms_norm(**{**t, "x": x3}, residual_out=x3, y=y3)
    assert torch.equal(x3, want_r) and torch.equal(y3, want_y)


@pytest.mark.parametrize("H", [2048, 7168])
def test_it_is_add_rms_norm_without_its_own_parts(H):
    """No post_weight, no gate, scales of one: the sum of x and residual is that of mdc_add_rms_norm, bit by bit; so is all
    the rest up to 2048 columns, where both kernels add the squares in the same order."""
    t = {k: v.to(DEV) for k, v in make(9, H, BF, F32, BF, None, 1, BF, False, 11).items()}
    outs = []
    for call in (mdc.mdc_add_rms_norm, mdc.mdc_block_rms_norm):
        o = dict(residual_out=torch.empty_like(t["residual"]), y=torch.empty_like(t["x"]),
                 q=torch.empty((9, H), device=DEV).to(E4M3), q_scale=torch.empty((9, H // 128), device=DEV))
        call(t["x"], t["weight"], residual=t["residual"], **o)
        outs.append(o)
    for k in outs[0] if H <= 2048 else ["residual_out"]:
        assert torch.equal(outs[0][k].view(torch.uint8), outs[1][k].view(torch.uint8)), k


def test_streams_and_graphs():
    t = {k: v.to(DEV) for k, v in make(40, 1024, BF, F32, BF, "wide", 10, BF, True, 12).items()}
    out = lambda: dict(residual_out=torch.empty_like(t["residual"]), y=torch.empty_like(t["x"]),  # noqa: E731
                       q=torch.empty((40, 1024), device=DEV).to(E4M3), q_scale=torch.empty((40, 8), device=DEV))
    a, b = out(), out()
    call = mdc.prepare_block_rms_norm(**t, **a, gate_every=10)
    call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mdc.mdc_block_rms_norm(**t, **b, gate_every=10)
    torch.cuda.synchronize()
    for k in a:
        assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mdc.mdc_block_rms_norm(**t, **b, gate_every=10)
    for rep in range(3):
        t["x"].copy_(torch.randn((40, 1024), device=DEV))
        b["y"].zero_()
        graph.replay()
        call()
        torch.cuda.synchronize()
        for k in a:
            assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), (rep, k)


def test_more_rows_than_threads_fit_a_dimension():
    """2^20 + 3 rows of 8: the second row of the grid."""
    rows = (1 << 20) + 3
    x = torch.randn((rows, 8), device=DEV).to(BF)
    gate = torch.randn((-(-rows // 1000), 8), device=DEV)
    out = torch.empty((rows, 8), device=DEV)
    mdc.mdc_block_rms_norm(x, gate=gate, gate_every=1000, residual_out=out)
    want = x.float() * gate[torch.arange(rows, device=DEV) // 1000]
    assert torch.equal(out, want)
