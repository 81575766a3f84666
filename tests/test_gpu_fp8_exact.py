"""The fp8 products on operands whose products and sums fp32 holds exactly: y is then known bit by bit, so that an error of a
scale, a missing k or a wrong block shows wherever it is."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_route_histogram_amd as mdc  # noqa: E402
from oracle import ops64 as O  # noqa: E402
from tests.test_gpu_fp8 import BF, DEV, E4M3, GROUP, HALF, group_max, np64  # noqa: E402


def small_codes(g, *shape):
    return torch.randint(-2, 3, shape, generator=g).to(E4M3)


def powers(g, lo, hi, *shape):
    return torch.exp2(torch.randint(lo, hi + 1, shape, generator=g).float())


def widened(codes, scales):
    return O.fp8_widen(np64(codes.float()), np64(scales))


def check_exact(counts, n, k, capacity=None, nums=True, seed=0):
    """Codes of 0, 1 and 2: no product lies 2^-13 below another, so an instruction loses nothing.  Scales of 2^-2 to 2^2 on
    either side: every sum is a multiple of 2^-4 and at most 4 * 2^4 k, which is below 2^24 such multiples for k < 2^14."""
    assert k < 2 ** 14
    used = min(sum(counts), capacity if capacity is not None else sum(counts))
    capacity = capacity if capacity is not None else used
    g = torch.Generator().manual_seed(seed)
    L, nk, nb = len(counts), -(-k // 128), -(-n // 128)
    a, sa = small_codes(g, capacity, k), powers(g, -2, 2, capacity, nk)
    w, sw = small_codes(g, L, n, k), powers(g, -2, 2, L, nb, nk)
    cnt = torch.tensor(counts, dtype=torch.int64)
    y = torch.full((capacity, n), 3.0, dtype=BF, device=DEV)
    mdc.mdc_gmm_fp8(a.to(DEV), sa.to(DEV), cnt.to(DEV) if nums else None, w.to(DEV), sw.to(DEV), y)
    torch.cuda.synchronize()
    left, real = used, []
    for c in counts:
        real.append(min(c, left))
        left -= real[-1]
    want = O.grouped(widened(a[:used], sa[:used]), widened(w, sw), real)
    got = y.cpu()
    assert (got[used:] == 3).all()
    # want is an fp32 value, so its rounding to bf16 is the only one
    wrong = got[:used] != torch.from_numpy(want).float().to(BF)
    assert not wrong.any(), (int(wrong.sum()), wrong.nonzero()[:5].tolist())


@pytest.mark.parametrize("rows", [1, 7, 16, 17, 32, 33, 64, 100, 129, 256, 300, 520])
@pytest.mark.parametrize("n,k", [(256, 384), (136, 2000)])
def test_rows_of_one_expert(rows, n, k):
    check_exact([rows], n, k, seed=rows + k)


@pytest.mark.parametrize("k", [16, 112, 128, 144, 256, 400, 640, 1152, 1280, 2000, 128 * 35 + 16, 128 * 101 + 48])
def test_lengths_of_k(k):
    check_exact([5, 40, 0, 29, 300], 136, k, seed=k)


@pytest.mark.parametrize("n", [8, 24, 128, 136, 248, 256, 264, 520, 1160])
def test_widths(n):
    check_exact([20, 0, 90], n, 528, seed=n)


# with 256 CUs: tiles of 256, 256, 128, 128, 64, 64 and 32 rows, and few rows an expert beside them
@pytest.mark.parametrize("counts", [
    [1000, 256, 700, 480, 380], [2048, 1900, 300, 40, 5], [500, 400, 380, 300, 128, 230, 90], [1024, 1000],
    [300, 400, 210, 90, 60], [600, 0, 200], [100, 40, 60, 32, 33, 3]])
def test_tiles(counts):
    check_exact(counts, 4104, 400, seed=len(counts))


@pytest.mark.parametrize("counts,capacity", [([300, 20], 400), ([3, 0, 32, 9], 44)])
def test_the_widths_of_a_layer(counts, capacity):
    check_exact(counts, 4096, 7168, capacity=capacity, seed=7)


def test_many_experts():
    counts = np.random.default_rng(1).integers(0, 5, 1000).tolist()
    counts[500] = 77
    check_exact(counts, 64, 272, capacity=sum(counts) + 3, seed=2)


def test_one_matrix_without_counts():
    check_exact([70], 512, 512, nums=False, seed=1)


def check_ffn_elements(counts, H, N, capacity, seed=0):
    """Each element of the FFN's y, from fp8 rows.  h is exact as above; g is then off by the rounding of fp32's
    operations only, so that its codes are known but for those whose value lies that near a border."""
    g = torch.Generator().manual_seed(seed)
    L, I = len(counts), N // 2
    given, counts, used = counts, [], 0
    for c in given:   # negative counts are none, rows past the capacity are not there
        counts.append(min(max(c, 0), capacity - used))
        used += counts[-1]
    # sums of h: multiples of 2^-7, at most 4 H 2^-4
    q, qs = small_codes(g, capacity, H), powers(g, -2, 0, capacity, H // 128)
    w1, s1 = small_codes(g, L, N, H), powers(g, -5, -4, L, N // 128, H // 128)
    w2, s2 = small_codes(g, L, H, I), powers(g, -2, 2, L, H // 128, I // 128)
    shape = mdc.Shape(1, 0, capacity, H, 1, L, capacity)
    ws = torch.full((mdc.mdc_ffn_fp8_workspace(shape, N),), 0x5A, dtype=torch.uint8, device=DEV)
    y = torch.full((capacity, H), 3.0, dtype=BF, device=DEV)
    mdc.mdc_ffn_fp8_quant_input(shape, N, *[t.to(DEV) for t in (q, qs, torch.tensor(given), w1, s1, w2, s2)], y, ws)
    torch.cuda.synchronize()
    h = O.grouped(widened(q[:used], qs[:used]), widened(w1, s1), counts)
    gate, up = h[:, :I], h[:, I:]
    v = gate / (1 + np.exp(-gate)) * up
    # silu: the exponential's argument times 1 / ln 2 (two roundings), the exponential and the reciprocal of 2^-23
    # each, the sum and two products; then the quotient by amax, which is off by as much, in four roundings
    rel = (2 * np.abs(gate).max() + 2 + 2 + 3) * 2.0 ** -24
    codes, scale = O.fp8_quant(v)
    wide = O.fp8_widen(np.ones_like(v), scale)
    value = v / np.where(wide > 0, wide, 1)
    off = (2 * rel + 8 * 2.0 ** -24) * np.abs(value)
    unsure = np.maximum(np.abs(O.e4m3_round(np.clip(value + off, -448, 448)) - codes),
                        np.abs(O.e4m3_round(np.clip(value - off, -448, 448)) - codes)) * wide
    v2, vw = codes * wide, widened(w2, s2)
    want = O.grouped(v2, vw, counts)
    size = O.grouped(np.abs(v2), np.abs(vw), counts)
    tol = HALF * np.abs(want) + GROUP * O.grouped(group_max(v2), group_max(vw), counts) + \
        O.grouped(unsure, np.abs(vw), counts) + (rel + (16 + 2 * (I // 128)) * 2.0 ** -23) * size
    err = np.abs(np64(y[:used]) - want)
    assert np.all(err <= tol), (err / np.maximum(tol, 1e-30)).max()
    assert (y[used:] == 3).all()
    # the bound is a sharp one: an error of 5% in an element is past it for most of them
    assert np.mean(0.05 * np.abs(want) > tol) > 0.5


@pytest.mark.parametrize("counts,H,N,capacity", [
    ([3, 0, 17], 256, 512, 64), ([2, 0, 17, 32] * 4, 256, 1024, 240), ([31, 33], 1664, 512, 64),
    ([70], 384, 512, 128), ([64, 65, 1, 0], 512, 768, 200), ([520], 1152, 1280, 600), ([300, 5, 129], 256, 512, 434)])
def test_elements_of_the_ffn(counts, H, N, capacity):
    check_ffn_elements(counts, H, N, capacity, seed=H + N)


@pytest.mark.parametrize("counts", [[1024, 1000], [900, 600, 200, 300, 40], [250, 200, 130], [100, 60], [20, 9] * 8])
def test_elements_of_the_ffn_over_its_tiles(counts):
    check_ffn_elements(counts, 128, 8192, sum(counts) + 9, seed=sum(counts))


@pytest.mark.parametrize("counts,capacity", [([20, -3, 30, 2 ** 40, 7], 70), ([30, 5, 9], 33), ([300, 50, -5, 900], 400)])
def test_ffn_counts_past_the_capacity(counts, capacity):
    check_ffn_elements(counts, 256, 512, capacity, seed=capacity)
