"""mdc_gmm_int8 with as many experts as its table holds: the instance with less LDS for the tiles, in each of its ways, bit by
bit as in the tests beside this one."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from tests.test_gpu_gmm_int8 import BF, F32, check  # noqa: E402

L = 2048


def way(counts, n, k):
    """The tiles that the plan takes for the experts of more than 32 rows: (rows of a tile, k-blocks over the wavefronts)."""
    G = -(-torch.cuda.get_device_properties(0).multi_processor_count // 8) * 8
    nk = -(-k // 128)
    tiles = {rows: sum(-(-c // rows) for c in counts if c > 32) for rows in (256, 128, 64, 32)}
    cost = {(rows, False): c * -(-tiles[rows] * -(-n // 256) // G) * nk
            for rows, c in ((256, 200), (128, 120), (64, 80), (32, 60))}
    cost[(64, True)] = -(-tiles[64] * -(-n // 64) // G) * (24 * nk + 200)
    return min(cost, key=cost.get)   # (the first of equals)


def counts_of(size, few):
    """One round of tiles of `size` rows x two tiles of columns, by an expert of many tiles and some of three, thin ones between."""
    G = -(-torch.cuda.get_device_properties(0).multi_processor_count // 8) * 8
    rng = np.random.default_rng(size)
    counts = [0] * L
    for e in rng.choice(L, 60, replace=False):
        counts[e] = int(rng.integers(1, 33))
    m = G // 2 if not few else 9
    for i, e in enumerate((0, 3, 1611, 1612, 1800, L - 1)):
        counts[e] = 3 * size - 5 * i if i else (m - 15) * size - 7
    if few:
        counts[0] = size + 1
    return counts


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size,split,n,k", [(32, False, 264, 144), (64, False, 264, 144), (128, False, 264, 144),
                                            (256, False, 264, 144), (128, False, 264, 400), (64, True, 72, 1168)])
def test_each_way(size, split, n, k, dtype):
    counts = counts_of(size, few=split)
    assert way(counts, n, k) == (size, split)
    check(counts, n, k, capacity=sum(counts) + 2, dtype=dtype, seed=size)


@pytest.mark.parametrize("experts", [1611, 1612, 1613])
def test_on_both_sides_of_the_tables_border(experts):
    """Ten bytes of LDS an expert: from about 1612 on the other instance."""
    rng = np.random.default_rng(experts)
    counts = [int(c) for c in rng.integers(0, 3, experts)]
    counts[7], counts[-1] = 300, 40
    check(counts, 72, 272, capacity=sum(counts), seed=experts)
