"""int8 product, norms around a block and expert layer where offsets pass 32 bits: rows, experts and gates that lie past
4 GB give, bit by bit, what the same rows and experts give in a small problem."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_route_histogram_amd as mdc  # noqa: E402

DEV = "cuda"
BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8


def codes(*shape):
    """int8 values, the same for the same shape."""
    g = torch.Generator(DEV).manual_seed(sum(shape))
    return torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=I8)


def product(a, sa, counts, w, sw, dtype):
    y = torch.full((a.shape[0], w.shape[-2]), 3.0, dtype=dtype, device=DEV)
    mdc.mdc_gmm_int8(a, sa, torch.tensor(counts, device=DEV), w, sw, y)
    return y


@pytest.mark.parametrize("dtype", [BF, F32])
def test_product_of_far_rows(dtype):
    k, n, rows = 8176, 520, 700_000   # a: 5.7 GB
    a, w = codes(rows, k), codes(3, n, k)
    sa, sw = torch.rand(rows, device=DEV) + 0.5, (torch.rand((3, n), device=DEV) + 0.5) * 1e-4
    counts = [rows - 100, 60, 9]
    y = product(a, sa, counts, w, sw, dtype)
    assert a.numel() > 2 ** 32 and (y[rows - 31:] == 3).all()
    for lo, hi, e in ((0, 40, 0), (2 ** 32 // k - 20, 2 ** 32 // k + 300, 0), (rows - 130, rows - 100, 0), (rows - 100, rows - 40, 1),
                      (rows - 40, rows - 31, 2)):
        small = product(a[lo:hi].clone(), sa[lo:hi].clone(), [hi - lo], w[e:e + 1].clone(), sw[e:e + 1].clone(), dtype)
        assert torch.equal(y[lo:hi], small), (lo, hi)


def test_outputs_past_32_bits():
    n, k, rows = 4104, 16, 550_000   # y: 2.26e9 values, 9 GB in fp32
    a, w = codes(rows, k), codes(1, n, k)
    sa, sw = torch.rand(rows, device=DEV) + 0.5, torch.rand((1, n), device=DEV) + 0.5
    y = product(a, sa, [rows - 3], w, sw, F32)
    assert y.numel() > 2 ** 31 and (y[rows - 3:] == 3).all()
    for lo in (0, 2 ** 30 // n - 50, 2 ** 31 // n - 50, rows - 103):
        small = product(a[lo:lo + 100].clone(), sa[lo:lo + 100].clone(), [100], w, sw, F32)
        assert torch.equal(y[lo:lo + 100], small), lo


def test_product_of_far_experts():
    L, n, k = 600, 1040, 8192   # w: 5.1 GB
    w, sw = codes(L, n, k), (torch.rand((L, n), device=DEV) + 0.5) * 1e-4
    assert w.numel() > 2 ** 32
    counts = [0] * L
    far = {0: 3, 503: 40, 504: 20, 598: 300, 599: 5}
    for e, c in far.items():
        counts[e] = c
    rows = sum(counts)
    a, sa = codes(rows, k), torch.rand(rows, device=DEV) + 0.5
    y, at = product(a, sa, counts, w, sw, BF), 0
    for e, c in far.items():
        small = product(a[at:at + c].clone(), sa[at:at + c].clone(), [c], w[e:e + 1].clone(), sw[e:e + 1].clone(), BF)
        assert torch.equal(y[at:at + c], small), e
        at += c


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("T", [1, 20])
def test_layer_of_far_experts(fmt, T):
    L, N, H, K = 270, 4096, 8192, 3
    call, size = (mdc.mdc_moe, mdc.mdc_moe_workspace) if fmt == "int8" else (mdc.mdc_moe_fp8, mdc.mdc_moe_fp8_workspace)
    if fmt == "int8":
        w1, w2 = codes(L, N, H), codes(L, H, N // 2)   # 9 and 4.5 GB
        s1, s2 = (torch.rand(s, device=DEV) * 1e-4 + 1e-4 for s in ((L, N), (L, H)))
    else:
        # e4m3 of exponents that make no NaN, any sign
        w1, w2 = (codes(*s).view(torch.uint8).bitwise_and(0xBF).view(torch.float8_e4m3fn) for s in ((L, N, H), (L, H, N // 2)))
        s1, s2 = (torch.rand(s, device=DEV) * 1e-3 + 1e-3 for s in ((L, N // 128, H // 128), (L, H // 128, N // 256)))
    assert w2.numel() > 2 ** 32
    x = torch.randn((T, H), device=DEV).to(BF)
    used = [1, 130, 257, 268, 269]
    pick = torch.stack([torch.randperm(len(used))[:K] for _ in range(T)])
    ids, scales = torch.tensor(used)[pick].int().to(DEV), torch.rand((T, K), device=DEV) + 0.1

    def run(experts, ids, *w):
        sh = mdc.Shape(1, 0, T, H, K, experts, 0)
        out = torch.zeros((T, H), dtype=BF, device=DEV)
        ws = torch.empty(size(sh, N), dtype=torch.uint8, device=DEV)
        call(sh, N, x, None, None, ids, scales, *w, out, ws)
        return out

    got = run(L, ids, w1, s1, w2, s2)
    at = torch.tensor(used, device=DEV)
    want = run(len(used), pick.int().to(DEV), *((w.view(torch.uint8)[at].view(w.dtype) if w.dtype != F32 else w[at])
                                                for w in (w1, s1, w2, s2)))
    assert torch.isfinite(got.float()).all() and got.any(1).all() and torch.equal(got, want)


@pytest.mark.parametrize("quant", ["int8", "fp8"])
def test_norms_of_far_rows(quant):
    rows, H = 68_000, 32768   # 2.2e9 elements, 4.5 GB each of x, gate, residual, y
    g = torch.Generator(DEV).manual_seed(1)
    new = lambda *s: torch.randn(s, generator=g, device=DEV, dtype=BF)  # noqa: E731
    x, gate, res, post, weight = new(rows, H), new(rows, H), new(rows, H), new(H), new(H)
    assert x.numel() > 2 ** 31

    def run(x, gate, res):
        n = x.shape[0]
        q = torch.empty((n, H), dtype=I8 if quant == "int8" else torch.uint8, device=DEV)
        qs = torch.empty((n,) if quant == "int8" else (n, H // 128), device=DEV)
        y = torch.empty_like(x)
        mdc.mdc_block_rms_norm(x, weight, post_weight=post, gate=gate, gate_act="tanh", residual=res, residual_out=res, y=y, q=q,
                               q_scale=qs)
        return y, q, qs, res

    spots = (0, 2 ** 30 // H - 2, 2 ** 31 // H - 2, rows - 4)
    small = [run(*(t[lo:lo + 4].clone() for t in (x, gate, res))) for lo in spots]
    big = run(x, gate, res)
    for lo, want in zip(spots, small):
        for b, w in zip(big, want):
            assert torch.equal(b[lo:lo + 4], w), lo
