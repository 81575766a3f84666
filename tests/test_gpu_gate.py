"""mdc_gate against the 64-bit oracle: ids equal, weights to fp32 rounding."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_route_histogram_amd as mdc  # noqa: E402
from oracle import ops64 as O  # noqa: E402

DEV = "cuda"


def run(logits, bias, topk, stream=None, guard=3, special=(0, 0), **kw):
    T, n = logits.shape
    shape = mdc.Shape(1, 0, T, 8, topk, n - sum(special), 0, zero_experts=special[0], copy_experts=special[1])
    ids = torch.full((T + guard, topk), -77, dtype=torch.int32, device=DEV)
    w = torch.full((T + guard, topk), -77.0, device=DEV)
    mdc.mdc_gate(shape, logits.to(DEV), None if bias is None else bias.to(DEV), ids, w, stream=stream, **kw)
    torch.cuda.synchronize()
    assert (ids[T:] == -77).all() and (w[T:] == -77).all()   # rows behind the last token are left as they were
    return ids[:T].cpu().numpy(), w[:T].cpu().numpy()


def check(logits, bias, topk, **kw):
    got_i, got_w = run(logits, bias, topk, **kw)
    kw.pop("special", None)
    want_i, want_w = O.gate(logits.double().numpy(), None if bias is None else bias.double().numpy(), topk, **kw)
    assert np.array_equal(got_i, want_i), np.argwhere(got_i != want_i)[:5]
    # exp's argument is off by |z| 2^-24, a sum of at most 2048 / 64 + 6 terms per lane and wave by as many roundings
    z = logits.double().numpy()
    z = z[np.isfinite(z)]
    span = float(min(np.abs(z).max() * 2, 90)) if z.size else 0.0
    rel = (3 * span + 64) * 2.0 ** -24
    assert np.all(np.abs(got_w - want_w) <= rel * np.abs(want_w) + 1e-37 * kw.get("scale", 1.0)), \
        np.abs(got_w / want_w - 1).max()


def make(T, n, dtype, seed, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn((T, n), generator=g)).to(dtype), 0.1 * torch.randn((n,), generator=g)


SIZES = [(1, 1, 1), (1, 8, 2), (3, 64, 8), (33, 65, 16), (5, 128, 8), (7, 144, 6), (32, 256, 8), (9, 257, 3),
         (4, 512, 8), (3, 1000, 16), (2, 2048, 16), (4096, 64, 6), (4099, 144, 16), (4097, 250, 8)]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,n,k", SIZES)
def test_gate_sizes(T, n, k, dtype, score):
    if T > 4000 and dtype == torch.float16:
        pytest.skip("large sizes in two types")
    logits, bias = make(T, n, dtype, 7 * n + k)
    check(logits, bias if (n + k) % 2 else None, k, score=score, renormalise=(T % 2 == 1), scale=2.5)


@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,n,k,groups,topk_groups,group_top", [
    (5, 256, 8, 8, 4, 2), (4100, 256, 8, 8, 4, 2), (3, 144, 6, 9, 3, 1), (2, 64, 4, 64, 5, 1), (7, 2048, 16, 16, 2, 2),
    (4096, 96, 2, 16, 1, 2), (3, 30, 5, 3, 3, 2)])
def test_gate_groups(T, n, k, groups, topk_groups, group_top, score, with_bias):
    logits, bias = make(T, n, torch.float32, n + groups)
    check(logits, bias if with_bias else None, k, score=score, groups=groups, topk_groups=topk_groups,
          group_top=group_top)


@pytest.mark.parametrize("T", [6, 5000])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_gate_ties_go_to_the_lowest_id(T, score, with_bias):
    g = torch.Generator().manual_seed(3)
    logits = torch.randint(-2, 3, (T, 128), generator=g).float()   # five values: every choice is a tie
    logits[0] = 0.0
    logits[1, ::2] = -0.0
    logits[1, 1::2] = 0.0
    bias = torch.randint(0, 2, (128,), generator=g).float() / 4 if with_bias else None
    check(logits, bias, 8, score=score)
    check(logits, bias, 8, score=score, groups=8, topk_groups=3, group_top=2)


@pytest.mark.parametrize("T", [64, 4096])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gate_keys_closer_than_fp32_can_tell(T, score):
    """Keys that differ by less than an fp32 step of a probability are ordered as in 64 bits."""
    g = torch.Generator().manual_seed(5)
    base = torch.randn((T, 1), generator=g)
    logits = base + 1e-6 * torch.randn((T, 256), generator=g)
    bias = 1e-8 * torch.randn((256,), generator=g)
    check(logits, bias, 8, score=score)
    check(logits, None, 8, score=score, groups=8, topk_groups=4)
    check(logits, bias, 8, score=score, groups=8, topk_groups=4, group_top=2)


@pytest.mark.parametrize("T", [40, 4104])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 8])
def test_gate_ids_that_are_off(T, score, groups):
    """NaN and -inf turn ids off, rows with fewer than K left get -1, +inf is the largest finite value."""
    logits, bias = make(T, 64, torch.float32, 11)
    inf, nan = float("inf"), float("nan")
    logits[0] = -inf
    logits[1] = nan
    logits[2, :] = -inf
    logits[2, 17] = -3.0
    logits[3, ::2] = nan
    logits[4, 5] = inf
    logits[5, [3, 9]] = inf
    logits[6, :] = -3.4028234663852886e38
    logits[7, :60] = -inf
    logits[8] = 3.4028234663852886e38
    for b in (None, bias):
        check(logits, b, 8, score=score, groups=groups, topk_groups=min(groups, 3))
        check(logits, b, 8, score=score, groups=groups, topk_groups=min(groups, 3), renormalise=False)
    bias[7] = -inf
    bias[9] = nan
    bias[11] = inf
    check(logits, bias, 8, score=score, groups=groups, topk_groups=min(groups, 3))


def test_gate_zero_and_copy_experts_are_among_the_ids():
    logits, bias = make(33, 144, torch.bfloat16, 2)
    check(logits, bias, 8, special=(8, 8))


def test_gate_small_probabilities_renormalise():
    """The chosen ids may be ones whose softmax probability is below fp32's range."""
    logits = torch.zeros((2, 64))
    logits[:, 0] = 300.0
    bias = torch.zeros(64)
    bias[1:9] = 10.0
    check(logits, bias, 8)


def test_gate_is_repeatable_on_another_stream_and_in_a_graph():
    T, n, k = 300, 256, 8
    logits, bias = make(T, n, torch.float32, 21)
    lg, b = logits.to(DEV), bias.to(DEV)
    shape = mdc.Shape(1, 0, T, 8, k, n, 0)
    want_i, want_w = run(logits, bias, k, score="sigmoid", groups=8, topk_groups=4, group_top=2)
    ids = torch.empty((T, k), dtype=torch.int32, device=DEV)
    w = torch.empty((T, k), device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mdc.mdc_gate(shape, lg, b, ids, w, score="sigmoid", groups=8, topk_groups=4, group_top=2)
    s.synchronize()
    assert np.array_equal(ids.cpu().numpy(), want_i) and np.array_equal(w.cpu().numpy(), want_w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mdc.mdc_gate(shape, lg, b, ids, w, score="sigmoid", groups=8, topk_groups=4, group_top=2)
    for rep in range(3):
        new, _ = make(T, n, torch.float32, 30 + rep)
        lg.copy_(new)
        ids.fill_(-5)
        graph.replay()
        torch.cuda.synchronize()
        want = run(new, bias, k, score="sigmoid", groups=8, topk_groups=4, group_top=2)
        assert np.array_equal(ids.cpu().numpy(), want[0]) and np.array_equal(w.cpu().numpy(), want[1])
