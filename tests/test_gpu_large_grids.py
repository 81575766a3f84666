"""The gate and the norm on more rows than one dimension of a grid takes threads for (2^32), and on rows whose int8 scale
has no finite reciprocal."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_route_histogram_amd as mdc  # noqa: E402

DEV = "cuda"


def test_norm_of_more_than_2_to_26_rows():
    rows, H = 2 ** 26 + 5, 8   # 64 threads a row
    x = torch.empty((rows, H), dtype=torch.bfloat16, device=DEV)
    part = torch.randn((2 ** 20 + 7, H), device=DEV).to(torch.bfloat16)
    for at in range(0, rows, part.shape[0]):
        n = min(part.shape[0], rows - at)
        x[at:at + n] = part[:n]
    y = torch.full((rows + 1, H), 3.0, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    mdc.mdc_add_rms_norm(x, w, y=y[:rows])
    want = torch.empty_like(part)
    mdc.mdc_add_rms_norm(part, w, y=want)
    for at in range(0, rows, part.shape[0]):
        n = min(part.shape[0], rows - at)
        assert torch.equal(y[at:at + n], want[:n]), at
    assert (y[rows:] == 3).all()
    f = part[:1000].double()
    f = f / (f.square().mean(1, keepdim=True) + 1e-6).sqrt()
    # bf16's half step, and of fp32 the sum of eight squares (4 after the root), root, quotient, two products
    assert ((want[:1000].double() - f).abs() <= (2.0 ** -8 + 9 * 2.0 ** -23) * f.abs()).all()


def test_gate_of_more_than_2_to_28_tokens():
    T = 2 ** 28 + 3   # 16 lanes a token
    logits = torch.empty((T, 2), dtype=torch.bfloat16, device=DEV)
    part = torch.randint(-3, 4, (2 ** 20 + 11, 2), device=DEV).to(torch.bfloat16)
    for at in range(0, T, part.shape[0]):
        n = min(part.shape[0], T - at)
        logits[at:at + n] = part[:n]
    ids = torch.full((T + 1, 1), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T + 1, 1), -7.0, device=DEV)
    mdc.mdc_gate(mdc.Shape(1, 0, T, 8, 1, 2, 0), logits, None, ids[:T], w[:T], scale=2.0)
    want = (part[:, 1] > part[:, 0]).int()[:, None]
    for at in range(0, T, part.shape[0]):
        n = min(part.shape[0], T - at)
        assert torch.equal(ids[at:at + n], want[:n]), at
    assert (w[:T] == 2).all() and (ids[T:] == -7).all() and (w[T:] == -7).all()


def test_int8_rows_of_tiny_values_keep_their_zeros():
    x = torch.zeros((3, 64), dtype=torch.bfloat16, device=DEV)
    x[0, 5] = 1e-40     # times 1 / sqrt(eps) = 1000: 127 / amax is past fp32
    x[1, 7] = -1e-30
    q = torch.full((3, 64), 9, dtype=torch.int8, device=DEV)
    s = torch.full((3,), 9.0, device=DEV)
    mdc.mdc_add_rms_norm(x, torch.ones(64, dtype=torch.bfloat16, device=DEV), q=q, q_scale=s, eps=1e-6)
    q = q.cpu()
    assert q[0, 5] > 0 and q[1, 7] == -127
    q[0, 5], q[1, 7] = 0, 0
    assert not q.any() and torch.isfinite(s).all() and s[2] == 0
