"""mdc_gate where the order of the choices is in doubt: neighbours that differ by one fp32 step of a logit, equal ones,
long runs of them, and rows that are not aligned for wide loads."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_route_histogram_amd as mdc  # noqa: E402
from oracle import ops64 as O  # noqa: E402
from tests.test_gpu_gate import DEV, check, make, run  # noqa: E402


def close_pairs(T, n, seed, run_of=2):
    """Each row holds runs of `run_of` logits one fp32 step apart, in a random order."""
    g = torch.Generator().manual_seed(seed)
    head = 1.5 * torch.randn((T, -(-n // run_of)), generator=g)
    rows = [head]
    for _ in range(run_of - 1):
        rows.append(torch.nextafter(rows[-1], torch.full_like(head, 9.0)))
    z = torch.cat(rows, 1)[:, :n]
    return torch.gather(z, 1, torch.rand((T, n), generator=g).argsort(1)).contiguous()


def check_groups(logits, k, score):
    """Four groups scored by their two largest, two open.  In a run of logits one step apart the sums of two pairs can be
    equal to first order (steps 0 + 3 and 1 + 2) and differ by the square of a step, 1e-22, which no 64-bit sum shows: an
    exponential and a division of one rounding (2^-53) each on either side and the sum's own leave 5 2^-53 of the score
    open.  Rows whose border is closer than that may open either group; all else is as in 64 bits."""
    kw = dict(score=score, groups=4, topk_groups=2, group_top=2)
    got, _ = run(logits, None, k, **kw)
    z = logits.double().numpy()
    want, _ = O.gate(z, None, k, **kw)
    size = z.shape[1] // 4
    for t in np.unique(np.argwhere(got != want)[:, 0]):
        p = 1 / (1 + np.exp(-z[t])) if score == "sigmoid" else np.exp(z[t] - z[t].max()) / np.exp(z[t] - z[t].max()).sum()
        sums = np.sort(p.reshape(4, size), 1)[:, -2:].sum(1)
        open_groups = np.unique(got[t] // size)
        closed = np.setdiff1d(np.arange(4), open_groups)
        assert len(open_groups) == 2 and sums[open_groups].min() >= sums[closed].max() * (1 - 5 * 2.0 ** -53), t
        live = np.flatnonzero(np.isin(np.arange(z.shape[1]) // size, open_groups))
        assert np.array_equal(got[t], live[np.argsort(-p[live], kind="stable")][:k]), t


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,n,k", [(5, 64, 1), (64, 256, 8), (4100, 256, 8), (4097, 128, 16), (4096, 60, 7), (9, 257, 16),
                                   (3, 2048, 16), (3, 520, 4), (4200, 17, 16), (50, 16, 16)])
@pytest.mark.parametrize("run_of", [2, 3, 9])
def test_neighbours_one_step_apart(T, n, k, run_of, score):
    logits = close_pairs(T, n, n + k, run_of)
    check(logits, None, k, score=score)                      # the order of the logits
    check(logits, torch.zeros(n), k, score=score)            # the order of the probabilities
    check(logits, 0.25 * torch.ones(n), k, score=score)
    if n % 4 == 0 and k <= n // 2:
        check_groups(logits, k, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,n", [(33, 256), (4100, 256), (4100, 64), (7, 1000)])
def test_equal_logits_of_16_bits(T, n, dtype, score):
    logits, bias = make(T, n, dtype, n)   # 16-bit logits: many are equal
    logits = (logits * 4).round() / 4
    check(logits, None, 8, score=score)
    check(logits, (bias * 8).round() / 8, 8, score=score)
    logits[:, ::7] = float("inf")
    check(logits, None, 8, score=score)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [40, 4100])
@pytest.mark.parametrize("offset", [1, 2])
def test_rows_that_are_not_aligned(T, dtype, offset):
    n, k = 256, 8
    logits, bias = make(T, n, dtype, 3)
    for aligned_bias in (True, False):
        flat = torch.empty(T * n + 8, dtype=dtype, device=DEV)
        flat[offset:offset + T * n] = logits.reshape(-1).to(DEV)
        fb = torch.empty(n + 8, device=DEV)
        at = 0 if aligned_bias else 1
        fb[at:at + n] = bias.to(DEV)
        want = run(logits, bias, k, score="sigmoid", groups=8, topk_groups=4, group_top=2)
        got = run(flat[offset:offset + T * n].view(T, n), fb[at:at + n], k, score="sigmoid", groups=8, topk_groups=4,
                  group_top=2)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_one_large_logit_and_infinite_biases():
    logits, bias = make(4100, 128, torch.float32, 9)
    logits[::3, 5] = 80.0     # the others' probabilities lie far below one step of the largest
    logits[1::3, 7] = -90.0
    for score in ("softmax", "sigmoid"):
        check(logits, None, 8, score=score, groups=4, topk_groups=3)
        check(logits, bias, 8, score=score)
    bias[[3, 4, 5]] = float("inf")
    bias[9] = -float("inf")
    check(logits, bias, 8, score="sigmoid")


def test_no_tokens():
    shape = mdc.Shape(1, 0, 0, 8, 2, 16, 0)
    e = torch.empty((0, 16), device=DEV)
    mdc.mdc_gate(shape, e, None, torch.empty((0, 2), dtype=torch.int32, device=DEV), torch.empty((0, 2), device=DEV))
    torch.cuda.synchronize()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,n,k,groups,topk_groups", [(5, 2040, 16, 8, 3), (4, 2048, 8, 2, 1), (4097, 250, 8, 5, 2),
                                                     (4096, 256, 8, 16, 4), (4100, 240, 4, 15, 15), (6, 1530, 9, 51, 2),
                                                     (4099, 16, 1, 16, 1), (3, 12, 12, 4, 4)])
def test_groups_of_whole_lanes_and_others(T, n, k, groups, topk_groups, score):
    logits, bias = make(T, n, torch.float32, n + groups)
    for top in (1, 2):
        if top <= n // groups:
            check(logits, bias, k, score=score, groups=groups, topk_groups=topk_groups, group_top=top)
    check(logits[:, :].bfloat16(), None, k, score=score, groups=groups, topk_groups=topk_groups, group_top=1)
