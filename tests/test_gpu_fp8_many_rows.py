"""The fp8 product on as many rows as its capacity can count, 2^31 - 1: the number of tiles, and every place, without a
32-bit overflow."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_route_histogram_amd as mdc  # noqa: E402

DEV = "cuda"
E4M3, BF = torch.float8_e4m3fn, torch.bfloat16


def test_product_of_2_to_31_rows():
    A, n, k = 2 ** 31 - 1, 8, 16
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GiB of GPU memory")
    g = torch.Generator().manual_seed(1)
    part = 2 ** 22 + 3
    pa = torch.randint(-2, 3, (part, k), generator=g).to(torch.int8)
    ps = torch.exp2(torch.randint(-2, 3, (part, 1), generator=g).float())
    w = torch.randint(-2, 3, (2, n, k), generator=g).to(torch.int8)
    # every product and sum is a multiple of 2^-2 and at most 2^8: the only rounding is that to bf16
    want = [((pa.double() @ w[e].double().t()) * ps.double()).float().to(BF).to(DEV) for e in range(2)]
    pa, ps, w = pa.float().to(E4M3).to(DEV), ps.to(DEV), w.float().to(E4M3).to(DEV)
    a = torch.empty((A, k), dtype=torch.uint8, device=DEV)
    sa = torch.empty((A, 1), device=DEV)
    y = torch.empty((A, n), dtype=BF, device=DEV)
    places = [(at, min(part, A - at)) for at in range(0, A, part)]
    for at, m in places:
        a[at:at + m] = pa.view(torch.uint8)[:m]
        sa[at:at + m] = ps[:m]
    ws = torch.ones((2, 1, 1), device=DEV)
    # one matrix; two experts, the second one's rows behind 2^31 - 301 others; likewise with few rows
    for nums in (None, [A - 300, 300], [A - 20, 20]):
        for at, m in places:
            y[at:at + m] = 7.0
        experts = 1 if nums is None else 2
        mdc.mdc_gmm_fp8(a, sa, None if nums is None else torch.tensor(nums, device=DEV), w[:experts], ws[:experts], y)
        last = A if nums is None else nums[0]   # rows of the first expert
        for at, m in places:
            head = max(0, min(m, last - at))
            assert torch.equal(y[at:at + head], want[0][:head]), (nums, at)
            assert torch.equal(y[at + head:at + m], want[1][head:m]), (nums, at)
    del a, sa, y
    torch.cuda.empty_cache()
