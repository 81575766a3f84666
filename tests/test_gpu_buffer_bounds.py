"""Loads past the end of a buffer descriptor whose offset stands in the scalar operand give zeros.

The products put the distance of a tile's rows there: rows past an expert's last, and k-blocks that a wavefront does not
have, are read as zeros by the descriptor's size alone.  Everything here lies inside one allocation.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

from combine_route_histogram_amd import probe  # noqa: E402

WORDS = 1 << 18


@pytest.mark.parametrize("bound,offset", [
    (4096, 0), (4096, 2048), (4096, 3584), (4096, 4080), (4096, 4096), (4096, 4112), (4096, 65536), (4096, (1 << 20) - 1024),
    (16, 0), (16, 16), (0, 0), (0, 2048), (1 << 19, (1 << 19) - 1024), (1 << 19, (1 << 19) - 16), (1 << 19, 1 << 19),
    (1 << 19, (1 << 19) + 8192)])
def test_zeros_from_the_bound_on(bound, offset):
    src = torch.arange(1, WORDS + 1, dtype=torch.int32, device="cuda")
    dst = torch.full((512,), -3, dtype=torch.int32, device="cuda")
    probe.bounded_read(src, bound, offset, dst, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    at = torch.arange(offset // 4, offset // 4 + 256)
    want = torch.where(at * 4 < bound, at + 1, 0).to(torch.int32)
    assert torch.equal(dst[:256].cpu(), want)   # into registers
    assert torch.equal(dst[256:].cpu(), want)   # into LDS
