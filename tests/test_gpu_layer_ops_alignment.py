"""Operands that are aligned as little as the header allows give, bit by bit, what aligned ones give."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_route_histogram_amd as mdc  # noqa: E402
from tests.test_gpu_fp8 import BF, DEV, E4M3  # noqa: E402
from tests.test_gpu_moe import FMT, weights  # noqa: E402

F32, I8 = torch.float32, torch.int8


def off(t, n=1):
    """A copy of t that starts n elements behind a 256-byte border."""
    if t is None:
        return None
    raw = torch.zeros(t.numel() + n, dtype=t.dtype, device=DEV)
    v = raw[n:].view(t.shape)
    v.copy_(t)
    assert v.data_ptr() % 16 == n * t.element_size() % 16
    return v


@pytest.mark.parametrize("dtype", [BF, torch.float16, F32])
@pytest.mark.parametrize("counts", [[1], [20, 3], [40, 0, 33], [300, 5, 700]])
def test_int8_product(counts, dtype):
    g = torch.Generator().manual_seed(len(counts))
    A, L, n, k = sum(counts), len(counts), 264, 656
    a = torch.randint(-127, 128, (A, k), generator=g, dtype=I8).to(DEV)
    w, sw = (t.to(DEV) for t in weights("int8", g, L, n, k, 0, 0))
    sa, nums = torch.rand(A, generator=g).to(DEV), torch.tensor(counts, device=DEV)
    y, z = (torch.zeros((A, n), dtype=dtype, device=DEV) for _ in range(2))
    mdc.mdc_gmm_int8(a, sa, nums, w, sw, y)
    mdc.mdc_gmm_int8(a, off(sa), off(nums), w, off(sw), z)
    assert y.any() and torch.equal(y, z)


@FMT
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("T", [1, 18])
def test_layer(fmt, gated, T):
    g = torch.Generator().manual_seed(T)
    E, N, H, K = 20, 512, 640, 4
    w1, s1 = (t.to(DEV) for t in weights(fmt, g, E, N, H, -5, -4))
    w2, s2 = (t.to(DEV) for t in weights(fmt, g, E, H, N // 2, -4, -1))
    x = torch.randn((T, H), generator=g).to(BF).to(DEV)
    logits = torch.randn((T, E), generator=g).to(BF).to(DEV) if gated else None
    bias = torch.randn(E, generator=g).to(DEV) if gated else None
    ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(T)]).int().to(DEV)
    scales, mask = torch.rand((T, K), generator=g).to(DEV), (torch.rand(T, generator=g) < 0.8).to(DEV)
    mask[0] = True
    call, size = (mdc.mdc_moe, mdc.mdc_moe_workspace) if fmt == "int8" else (mdc.mdc_moe_fp8, mdc.mdc_moe_fp8_workspace)
    shape, outs = mdc.Shape(1, 0, T, H, K, E, 0), []
    for f in (lambda t: None if t is None else t.clone(), off):
        out, i, s = torch.zeros((T, H), dtype=BF, device=DEV), f(ids), f(scales)
        ws = torch.empty(size(shape, N), dtype=torch.uint8, device=DEV)
        call(shape, N, x, f(logits), f(bias), i, s, w1, f(s1), w2, f(s2), out, ws, x_active_mask=f(mask))
        outs.append((out, i, s))
    for a, b in zip(*outs):
        assert a.any() and torch.equal(a, b)


@pytest.mark.parametrize("quant", ["int8", "fp8"])
@pytest.mark.parametrize("gate_dtype", [BF, F32])
@pytest.mark.parametrize("H", [8, 136, 2056, 5000])
def test_block_norm(H, gate_dtype, quant):
    g = torch.Generator().manual_seed(H)
    n = lambda *s: torch.randn(s, generator=g).to(DEV)  # noqa: E731
    x, res, w, gate = n(7, H).to(BF), n(7, H), n(H), n(7, 1).to(gate_dtype)
    outs = []
    for f, q_at in ((lambda t: t.clone(), 0), (off, 8)):
        q = off(torch.zeros((7, H), device=DEV).to(I8 if quant == "int8" else E4M3), q_at)
        s = f(torch.zeros((7,) if quant == "int8" else (7, -(-H // 128)), device=DEV))
        mdc.mdc_block_rms_norm(x, w, post_weight=w, gate=f(gate), gate_act="sigmoid", residual=res, q=q, q_scale=s)
        outs.append((q.view(torch.uint8), s))
    for a, b in zip(*outs):
        assert a.any() and torch.equal(a, b)
