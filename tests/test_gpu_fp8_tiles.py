"""The fp8 products over the sizes of tile that they choose between: many and few rows, experts that end inside a tile,
long k, more experts than the larger table of stages leaves room for, quantised blocks whole and split."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_route_histogram_amd as mdc  # noqa: E402
from tests.test_gpu_fp8 import BF, DEV, check_ffn, check_gmm, ffn_problem, problem  # noqa: E402


# With 256 CUs: tiles of 256 rows with ends of 124 to 256 rows and of 44 to 256, 128 with ends of 40 to 128 and 16 to
# 128, 64 with ends of 8 to 64 and 13 to 64, 32 rows.
@pytest.mark.parametrize("counts", [
    [1000, 256, 700, 480, 380], [500, 400, 380, 300, 128, 230, 90], [1024, 1000], [2048, 1900, 300, 40, 5],
    [300, 400, 210, 90, 60], [600, 0, 200], [128, 60, 77, 200, 1], [100, 40, 60, 32, 33]])
def test_gmm_tiles(counts):
    check_gmm(counts, 4104, 400, seed=len(counts))


@pytest.mark.parametrize("counts,n,k", [([100, 40, 60], 264, 128 * 35 + 16), ([600, 200], 4104, 128 * 19),
                                        ([1300, 700], 2056, 128 * 6 + 48), ([33], 8, 128 * 32), ([33], 8, 128 * 33)])
def test_gmm_tiles_of_long_rows(counts, n, k):
    check_gmm(counts, n, k, seed=k)


@pytest.mark.parametrize("last", [40, 32000])
def test_gmm_more_experts_than_three_stages_leave_room_for(last):
    counts = [0] * 850
    counts[3], counts[400], counts[849] = 7, 300, last
    check_gmm(counts, 136, 272, seed=last)


@pytest.mark.parametrize("counts", [
    [1024, 1000], [520, 500, 300], [900, 600, 200, 300, 40], [512, 480, 33, 7], [250, 200, 130], [100, 60]])
def test_ffn_tiles(counts):
    check_ffn(counts, 128, 8192, capacity=sum(counts) + 9, seed=sum(counts))


@pytest.mark.parametrize("counts,H,N,capacity", [
    ([5, 3], 128, 256, 300), ([2, 0, 17, 32] * 16, 256, 1024, 1000), ([33, 31, 32, 1] * 16, 128, 1024, 1600),
    ([32, 32], 1664, 512, 64), ([31, 33], 1664, 512, 64)])
def test_ffn_few_rows_whole_and_split_blocks(counts, H, N, capacity):
    check_ffn(counts, H, N, capacity, seed=H)


def test_ffn_many_experts():
    counts = [0] * 900
    counts[1], counts[450], counts[451], counts[899] = 3, 200, 40, 1
    check_ffn(counts, 128, 256, capacity=300, seed=1)


def test_gmm_values_outside_the_rows_in_use_do_not_matter():
    """NaN in rows behind the last expert, in the weights of experts without rows and in their scales."""
    counts = [0, 20, 0, 70, 0]
    a, sa, cnt, w, sw = problem(counts, 136, 272, 130, 1)
    args = [t.to(DEV) for t in (a, sa, cnt, w, sw)]
    want = torch.empty((130, 136), dtype=BF, device=DEV)
    mdc.mdc_gmm_fp8(*args, want)
    bad = [t.clone() for t in args]
    bad[0].view(torch.uint8)[90:] = 0x7F
    bad[1][90:] = float("nan")
    bad[3].view(torch.uint8)[[0, 2, 4]] = 0x7F
    bad[4][[0, 2, 4]] = float("inf")
    y = torch.full_like(want, 5.0)
    mdc.mdc_gmm_fp8(*bad, y)
    assert torch.equal(y[:90], want[:90]) and (y[90:] == 5).all()


@pytest.mark.parametrize("counts", [[3, 0, 20], [40, 300, 7]])
def test_gmm_on_a_stream_and_in_a_graph(counts):
    used = sum(counts)
    args = [t.to(DEV) for t in problem(counts, 264, 528, used + 5, 2)]
    want = torch.full((used + 5, 264), 5.0, dtype=BF, device=DEV)
    mdc.mdc_gmm_fp8(*args, want)
    y = torch.full_like(want, 5.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mdc.mdc_gmm_fp8(*args, y, stream=s)
    s.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mdc.mdc_gmm_fp8(*args, y)
    # the counts are read at each replay
    for new in (counts, [0] * len(counts), counts[::-1]):
        args[2].copy_(torch.tensor(new))
        want.fill_(5)
        y.fill_(5)
        mdc.mdc_gmm_fp8(*args, want)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_two_ffn_calls_at_once():
    """On two streams, each with its own workspace."""
    H, N, counts = 256, 512, [40, 100, 0, 3]
    shape = mdc.Shape(1, 0, 160, H, 1, len(counts), 160)
    x, cnt, *w = [t.to(DEV) for t in ffn_problem(counts, H, N, 160, 1)]
    size = mdc.mdc_ffn_fp8_workspace(shape, N)
    want = torch.zeros((160, H), dtype=BF, device=DEV)
    mdc.mdc_ffn_fp8(shape, N, x, cnt, *w, want, torch.empty(size, dtype=torch.uint8, device=DEV))
    torch.cuda.synchronize()
    runs = []
    for _ in range(2):
        s = torch.cuda.Stream()
        runs.append((s, torch.zeros_like(want), torch.empty(size, dtype=torch.uint8, device=DEV)))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, y, ws in runs:
            mdc.mdc_ffn_fp8(shape, N, x, cnt, *w, y, ws, stream=s)
    torch.cuda.synchronize()
    for _, y, _ws in runs:
        assert torch.equal(y, want)


def test_products_are_repeatable():
    """Sums are joined in one order, whichever workgroup comes first."""
    counts = [3, 200, 32, 0, 700, 17]
    args = [t.to(DEV) for t in problem(counts, 1160, 2000, sum(counts), 3)]
    first = torch.empty((sum(counts), 1160), dtype=BF, device=DEV)
    mdc.mdc_gmm_fp8(*args, first)
    for _ in range(5):
        y = torch.empty_like(first)
        mdc.mdc_gmm_fp8(*args, y)
        assert torch.equal(y, first)
    assert np.isfinite(first.float().cpu().numpy()).all()
