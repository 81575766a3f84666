"""mdc_moe and mdc_moe_fp8 at every number of columns that a workgroup of the second product may have, and with gates of
groups over many ids, against the 64-bit oracle as in the tests beside this one."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_route_histogram_amd as mdc  # noqa: E402
from oracle import ops64 as O  # noqa: E402
from tests.test_gpu_fp8 import DEV, np64  # noqa: E402
from tests.test_gpu_moe import FMT, Layer  # noqa: E402


def columns(H):
    """Output columns of a workgroup of the second product."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    return min(32, max(4, (-(-H // cus) + 3) // 4 * 4))


def sizes(cw):
    """Hidden sizes with that many columns: the least, and the last but one (a ragged last workgroup)."""
    all_of = [H for H in range(128, 8192 + 1, 128) if columns(H) == cw]
    return sorted({all_of[0], all_of[-2]}) if len(all_of) > 1 else all_of


@FMT
@pytest.mark.parametrize("cw", range(4, 33, 4))
def test_columns_of_a_workgroup(fmt, cw):
    """Each number of half blocks of eight columns, whole and with a half at the end; borders of w2's scales inside."""
    assert sizes(cw) or torch.cuda.get_device_properties(0).multi_processor_count != 256
    for H in sizes(cw):
        Layer(fmt, 5, 2, H, 512, 4, seed=H).check(shared=False)
        Layer(fmt, 18, 2, H, 256, 2, seed=H + 1).check()


@FMT
@pytest.mark.parametrize("H", [5120, 6144])
@pytest.mark.parametrize("T", [1, 16, 32])
def test_widths_in_use(fmt, H, T):
    Layer(fmt, T, 4, H, 768, 6, copy=1, seed=H + T).check()


@FMT
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("n,groups,open_groups,top", [
    (256, 8, 4, 2), (384, 8, 3, 2), (120, 5, 2, 1), (72, 3, 2, 2), (512, 4, 2, 2), (1000, 10, 5, 2), (2048, 64, 32, 2),
    (1984, 62, 9, 1)])
def test_gates_of_groups_over_many_ids(fmt, score, n, groups, open_groups, top):
    """Groups that are whole lanes and groups that are not (through LDS), 1 to 32 ids a lane: as mdc_gate, bit by bit."""
    K = 8
    for T in (1, 9):
        m = Layer(fmt, T, K, 128, 256, n // 2, zero=n // 4, copy=n - n // 2 - n // 4, seed=n + T)
        m.logits = 1.5 * torch.randn((T, n), generator=m.g)
        bias = (0.1 * torch.randn(n, generator=m.g)) if score == "sigmoid" else None
        how = dict(score=score, groups=groups, topk_groups=open_groups, group_top=top, scale=2.5)
        m.gate = dict(bias=None if bias is None else bias.to(DEV), **how)
        m.check(sharp=False)
        ids, _ = O.gate(np64(m.logits), None if bias is None else bias.numpy(), K, score, groups, open_groups, top, True, 2.5)
        assert (ids == m.got_ids.cpu().numpy()).all()
        want_i, want_w = torch.empty_like(m.got_ids), torch.empty_like(m.got_scales)
        mdc.mdc_gate(m.shape, m.logits.to(DEV), m.gate["bias"], want_i, want_w, **how)
        assert torch.equal(want_i, m.got_ids) and torch.equal(want_w, m.got_scales)
