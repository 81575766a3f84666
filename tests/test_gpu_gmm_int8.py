"""mdc_gmm_int8, bit by bit: the sum is exact, its conversion, two fp32 products and the last rounding are known."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_route_histogram_amd as mdc  # noqa: E402

DEV = "cuda"
BF, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def problem(counts, n, k, capacity, seed, lo=-128):
    g = torch.Generator().manual_seed(seed)
    L = len(counts)
    return (torch.randint(lo, 128, (capacity, k), generator=g, dtype=torch.int8),
            (torch.rand((capacity,), generator=g) + 0.5) * 1e-2, torch.tensor(counts, dtype=torch.int64),
            torch.randint(lo, 128, (L, n, k), generator=g, dtype=torch.int8),
            (torch.rand((L, n), generator=g) + 0.5) * 1e-2)


def real_counts(counts, capacity):
    out, left = [], capacity
    for c in counts:
        out.append(min(max(c, 0), left))
        left -= out[-1]
    return out


def expected(a, sa, counts, w, sw, dtype):
    """In fp32 as the formula rounds it."""
    out, at = [], 0
    for e, c in enumerate(counts):
        # products of 2^14 at most, fewer than 2^17 of them: float64 holds every sum
        acc = (a[at:at + c].double() @ w[e].double().t()).numpy()
        assert np.all(np.abs(acc) < 2 ** 31)
        v = acc.astype(np.int64).astype(np.float32) * sa[at:at + c].numpy()[:, None] * sw[e].numpy()[None, :]
        out.append(torch.from_numpy(v).to(dtype))
        at += c
    return torch.cat(out)


def check(counts, n, k, capacity=None, dtype=BF, seed=0, nums=True, data=None):
    real = real_counts(counts, capacity if capacity is not None else sum(counts))
    used = sum(real)
    capacity = capacity if capacity is not None else used
    a, sa, cnt, w, sw = data if data is not None else problem(counts, n, k, capacity, seed)
    y = torch.full((capacity, n), 3.0, dtype=dtype, device=DEV)
    mdc.mdc_gmm_int8(a.to(DEV), sa.to(DEV), cnt.to(DEV) if nums else None, w.to(DEV), sw.to(DEV), y)
    torch.cuda.synchronize()
    got = y.cpu()
    assert (got[used:] == 3).all()   # rows behind the last expert are left as they were
    want = expected(a, sa, real, w, sw, dtype)
    wrong = got[:used] != want
    assert not wrong.any(), (int(wrong.sum()), wrong.nonzero()[:5].tolist())


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 32, 33, 48, 49, 64, 65, 100, 128, 129, 191, 192, 193, 255, 256,
                                  257, 300, 512, 600])
def test_rows_of_one_expert(rows):
    check([rows], 264, 384, seed=rows)


@pytest.mark.parametrize("dtype", [BF, F16, F32])
@pytest.mark.parametrize("n", [8, 16, 24, 128, 136, 248, 256, 264, 520, 1160])
def test_widths_and_types(n, dtype):
    check([40, 0, 300, 7], n, 272, dtype=dtype, seed=n)


@pytest.mark.parametrize("k", [16, 32, 64, 112, 128, 144, 256, 400, 640, 1152, 2000, 128 * 35 + 16, 128 * 101 + 48])
def test_lengths_of_k(k):
    check([5, 40, 0, 29, 300], 136, k, seed=k)


@pytest.mark.parametrize("counts,capacity", [
    ([0, 0, 5, 0], 64), ([1] * 70, 70), ([3, 500, 0, 64, 65, 17], 700), ([100, 100, 100], 150), ([10, 20], 5),
    ([700, 1, 700], 1000), ([256, 512, 768], 1536), ([20, -3, 30, 2 ** 40, 7], 70)])
def test_experts(counts, capacity):
    check(counts, 136, 272, capacity=capacity, seed=len(counts))


@pytest.mark.parametrize("counts", [
    [1000, 256, 700, 480, 380], [2048, 1900, 300, 40, 5], [500, 400, 380, 300, 128, 230, 90], [1024, 1000],
    [300, 400, 210, 90, 60], [600, 0, 200], [100, 40, 60, 32, 33, 3], [24] * 9])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_tiles(counts, dtype):
    check(counts, 4104, 400, dtype=dtype, seed=len(counts))


# workgroups that pass from expert to expert, with up to eight and with nine k-blocks a wavefront
@pytest.mark.parametrize("counts,n,k", [([20, 32, 0, 17, 8] * 8, 1040, 1936), ([32, 5, 18] * 14, 520, 4112), ([31] * 70, 264, 1040)])
def test_streams_of_many_experts(counts, n, k):
    check(counts, n, k, seed=n)


# with 256 CUs: one or two rounds of tiles of 64 x 64, whose k-blocks go over the wavefronts, beside few rows an expert
@pytest.mark.parametrize("counts,n,k,capacity", [
    ([33], 1160, 2000, 33), ([64], 2056, 7168, 70), ([200, 5, 0, 65, 32], 328, 1040, 290), ([513], 136, 7184, 600),
    ([40] + [1, 0, 33] * 30, 72, 1936, 1100), ([100, 2 ** 40], 200, 4112, 300), ([1, 34, 2], 8, 1168, 37)])
@pytest.mark.parametrize("dtype", [BF, F16, F32])
def test_tiles_with_k_split(counts, n, k, capacity, dtype):
    check(counts, n, k, capacity=capacity, dtype=dtype, seed=k)


@pytest.mark.parametrize("counts,capacity", [([300, 20], 400), ([3, 0, 32, 9], 44), ([1, 1, 2], 4)])
def test_the_widths_of_a_layer(counts, capacity):
    check(counts, 4096, 7168, capacity=capacity, seed=7)


def test_many_experts():
    counts = np.random.default_rng(1).integers(0, 5, 2048).tolist()
    counts[500] = 77
    check(counts, 64, 272, capacity=sum(counts) + 3, seed=2)


@pytest.mark.parametrize("rows", [1, 70])
def test_one_matrix_without_counts(rows):
    check([rows], 512, 512, nums=False, seed=1)


@pytest.mark.parametrize("counts", [[0], [0, 0], [-4, 0]])
def test_no_rows(counts):
    a, sa, cnt, w, sw = (t.to(DEV) for t in problem(counts, 64, 128, 8, 3))
    y = torch.full((8, 64), 3.0, dtype=BF, device=DEV)
    mdc.mdc_gmm_int8(a, sa, cnt, w, sw, y)
    assert (y == 3).all()


def test_the_largest_sums():
    """K just below 2^17 of (-128)^2, the largest sum that there is, in both kinds of tiles."""
    k = 2 ** 17 - 16
    for rows in (3, 40):
        a, w = torch.full((rows, k), -128, dtype=torch.int8), torch.full((1, 8, k), -128, dtype=torch.int8)
        a[1] = 127
        data = (a, torch.full((rows,), 0.5), torch.tensor([rows]), w, torch.full((1, 8), 2.0 ** -20))
        check([rows], 8, k, data=data, dtype=F32)


def test_scales_that_are_zero_tiny_or_not_finite():
    a, sa, cnt, w, sw = problem([20, 40], 64, 128, 60, 8)
    sa[3], sa[4], sa[5], sa[30] = 0, 1e-42, float("nan"), float("inf")
    sw[0, 9] = 0
    y = torch.empty((60, 64), dtype=F32, device=DEV)
    mdc.mdc_gmm_int8(*[t.to(DEV) for t in (a, sa, cnt, w, sw)], y)
    want = expected(a, sa, [20, 40], w, sw, F32)
    assert torch.equal(torch.nan_to_num(y.cpu(), 7, 8, 9), torch.nan_to_num(want, 7, 8, 9))
    assert torch.isnan(y[5]).all() and torch.isfinite(y[[0, 1, 2, 6]]).all()


def test_streams_and_graphs():
    a, sa, cnt, w, sw = (t.to(DEV) for t in problem([40, 0, 300, 7], 520, 640, 347, 11))
    y, z = torch.zeros((347, 520), dtype=BF, device=DEV), torch.zeros((347, 520), dtype=BF, device=DEV)
    call = mdc.prepare_gmm_int8(a, sa, cnt, w, sw, y)
    call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mdc.mdc_gmm_int8(a, sa, cnt, w, sw, z)
    torch.cuda.synchronize()
    assert torch.equal(y, z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mdc.mdc_gmm_int8(a, sa, cnt, w, sw, z)
    for rep in range(3):
        a.copy_(torch.randint(-128, 128, a.shape, device=DEV, dtype=torch.int8))
        cnt.copy_(torch.tensor([[300, 40, 0, 7], [0, 347, 0, 0], [87, 87, 87, 86]][rep], device=DEV))
        z.zero_()
        graph.replay()
        call()
        torch.cuda.synchronize()
        assert torch.equal(y, z), rep


def test_the_rows_of_the_norm_and_of_the_quantised_dispatch_fit():
    """What the int8 norm writes goes in as it is, and the product is the int8 FFN's second one."""
    x, w = torch.randn((70, 512), device=DEV).to(BF), torch.ones(512, device=DEV, dtype=BF)
    q, s = torch.empty((70, 512), dtype=torch.int8, device=DEV), torch.empty(70, device=DEV)
    mdc.mdc_add_rms_norm(x, w, q=q, q_scale=s)
    _, _, _, m, ms = problem([70], 136, 512, 70, 12)
    y = torch.empty((70, 136), dtype=BF, device=DEV)
    mdc.mdc_gmm_int8(q, s, None, m.to(DEV)[0], ms.to(DEV), y)
    assert torch.equal(y.cpu(), expected(q.cpu(), s.cpu(), [70], m, ms, BF))
