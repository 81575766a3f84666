"""The norms around a block, the int8 product and the expert layer for a few tokens in a row, as a decode step uses them: the
block's output is normalised, weighed and added to the residual; the next norm's int8 rows go through the router's and the shared
expert's products, its bf16 rows and the router's logits through the experts; their sum enters the next block's norms."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_route_histogram_amd as mdc  # noqa: E402
from oracle import ops64 as O  # noqa: E402
from tests.test_gpu_fp8 import BF, DEV, HALF, np64  # noqa: E402
from tests.test_gpu_gmm_int8 import expected  # noqa: E402
from tests.test_gpu_moe import weights, widen  # noqa: E402

F32 = torch.float32


class Step:
    def __init__(self, fmt, T, H=512, N=768, E=24, K=4, seed=0):
        g = torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        d = lambda t: t.to(DEV)  # noqa: E731
        self.fmt, self.T, self.H, self.N, self.E = fmt, T, H, N, E
        self.shape = mdc.Shape(1, 0, T, H, K, E, 0)
        self.block, self.res = d(n(T, H).to(BF)), d(3 * n(T, H))
        self.post, self.pre, self.gate = (d((1 + 0.2 * n(H)).to(BF)) for _ in range(3))
        self.router, self.router_s = (d(t) for t in weights("int8", g, 1, E, H, 0, 0))
        self.router_s = self.router_s * 20     # logits that differ
        self.sh, self.sh_s = (d(t) for t in weights("int8", g, 1, H, H, 0, 0))
        self.w1, self.s1 = (d(t) for t in weights(fmt, g, E, N, H, -9, -8))
        self.w2, self.s2 = (d(t) for t in weights(fmt, g, E, H, N // 2, -9, -8))
        e = lambda *s, dt=BF: torch.full(s, 5, device=DEV).to(dt)  # noqa: E731
        self.res1, self.x, self.q, self.qs = e(T, H, dt=F32), e(T, H), e(T, H, dt=torch.int8), e(T, dt=F32)
        self.logits, self.shared, self.out = e(T, E, dt=F32), e(T, H), e(T, H)
        self.ids, self.scales = e(T, K, dt=torch.int32), e(T, K, dt=F32)
        self.res2, self.y2 = e(T, H, dt=F32), e(T, H)
        call, size = (mdc.mdc_moe, mdc.mdc_moe_workspace) if fmt == "int8" else (mdc.mdc_moe_fp8, mdc.mdc_moe_fp8_workspace)
        self.call = call
        self.ws = torch.empty(size(self.shape, N), dtype=torch.uint8, device=DEV)

    def run(self):
        mdc.mdc_block_rms_norm(self.block, self.pre, post_weight=self.post, gate=self.gate, residual=self.res,
                               residual_out=self.res1, y=self.x, q=self.q, q_scale=self.qs)
        mdc.mdc_gmm_int8(self.q, self.qs, None, self.router, self.router_s, self.logits)
        mdc.mdc_gmm_int8(self.q, self.qs, None, self.sh, self.sh_s, self.shared)
        self.call(self.shape, self.N, self.x, self.logits, None, self.ids, self.scales, self.w1, self.s1, self.w2, self.s2,
                  self.out, self.ws, shared_expert_x=self.shared)
        mdc.mdc_block_rms_norm(self.out, self.pre, post_weight=self.post, residual=self.res1, residual_out=self.res2, y=self.y2,
                               residual_scale=1.0, block_scale=0.5)

    def outputs(self):
        return [t.clone() for t in (self.res1, self.x, self.q, self.qs, self.logits, self.shared, self.ids, self.scales, self.out,
                                    self.res2, self.y2)]

    def check(self):
        """Each step from what the step before gave.

        Norms: a dozen fp32 roundings of terms that are at most |h|'s largest (below 20 here) leave h within 12 2^-24 of it, and v,
        where terms cancel, within 12 2^-24 20 times the inverse of the norm and a weight, together below 2: 3e-5.
        """
        n = np64
        h, v = O.block_rms_norm(n(self.block), n(self.post), n(self.gate)[None], max(self.T, 1), "none", n(self.res), n(self.pre),
                                1, 1, 1e-6, 1e-6)
        assert np.abs(n(self.res1) - h).max() < 1e-5 * np.abs(h).max()
        assert np.all(np.abs(n(self.x) - v) <= 1.01 * HALF * np.abs(v) + 1e-4)
        q, qs = self.q.cpu(), self.qs.cpu()
        assert np.all(np.abs(n(q) * n(qs)[:, None] - v) <= 0.51 * n(qs)[:, None])
        for m, s, y in ((self.router, self.router_s, self.logits), (self.sh, self.sh_s, self.shared)):
            assert torch.equal(y.cpu(), expected(q, qs, [self.T], m.cpu(), s.cpu(), y.dtype))
        ids, w = O.gate(n(self.logits), None, self.shape.topk)
        assert np.array_equal(ids, self.ids.cpu().numpy()) and np.allclose(w, n(self.scales), rtol=1e-5)
        x, want = n(self.x), n(self.scales).sum(1, keepdims=True) * n(self.shared)
        quant = (lambda u: (lambda c, s: c * s[:, None])(*O.int8_quant(u))) if self.fmt == "int8" else \
            (lambda u: O.fp8_widen(*O.fp8_quant(u)))
        for e in range(self.E):
            rows, k = np.nonzero(ids == e)
            if rows.size:
                hh = quant(x[rows]) @ widen(self.fmt, self.w1[e:e + 1].cpu(), self.s1[e:e + 1].cpu())[0].T
                a, b = hh[:, :self.N // 2], hh[:, self.N // 2:]
                want[rows] += n(self.scales)[rows, k][:, None] * \
                    (quant(a / (1 + np.exp(-a)) * b) @ widen(self.fmt, self.w2[e:e + 1].cpu(), self.s2[e:e + 1].cpu())[0].T)
        # bf16's rounding, and codes of g on the other side of a border: g is off by about 1e-6 of its value, so that 250e-6 of
        # the int8 codes differ by a step (1/127 of a row's largest, a fortieth of its norm) and 16e-6 of the e4m3 ones by
        # an eighth of their value: sqrt(250e-6) / 40 = 4e-4 and sqrt(16e-6) / 8 = 5e-4 of the norm, four times that allowed
        assert np.linalg.norm(n(self.out) - want) <= (2.0 ** -8 + 0.002) * np.linalg.norm(want)
        h, v = O.block_rms_norm(n(self.out), n(self.post), None, 1, "none", n(self.res1), n(self.pre), 0.5, 1, 1e-6, 1e-6)
        assert np.abs(n(self.res2) - h).max() < 1e-5 * np.abs(h).max()
        assert np.all(np.abs(n(self.y2) - v) <= 1.01 * HALF * np.abs(v) + 1e-4)


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("T", [1, 2, 5, 17, 32])
def test_a_step(fmt, T):
    s = Step(fmt, T, seed=T)
    s.run()
    torch.cuda.synchronize()
    s.check()


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_a_step_captured_and_replayed(fmt):
    s = Step(fmt, 7, seed=1)
    s.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for rep in range(3):
        s.block.copy_(torch.randn(s.block.shape, device=DEV))
        s.res.copy_(torch.randn(s.res.shape, device=DEV))
        for t in (s.res1, s.x, s.out, s.y2):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = s.outputs()
        s.check()
        s.run()
        torch.cuda.synchronize()
        for a, b in zip(got, s.outputs()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), rep


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
def test_steps_on_streams_side_by_side(fmt):
    """Two steps, each with its own workspace, at once; and two graphs that share one, in turn."""
    steps = [Step(fmt, T, seed=T) for T in (3, 20)]
    for s in steps:
        s.run()
    torch.cuda.synchronize()
    want = [s.outputs() for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    for s, st in zip(steps, streams):
        for t in (s.res1, s.x, s.out, s.y2):
            t.zero_()
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(8):
        for s, st in zip(steps, streams):
            with torch.cuda.stream(st):
                s.run()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        for a, b in zip(w, s.outputs()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    steps[0].ws = steps[1].ws
    graphs = []
    for s in steps:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            s.run()
    for i in (0, 1, 1, 0, 1, 0):
        steps[i].out.zero_()
        steps[i].y2.zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        for a, b in zip(want[i], steps[i].outputs()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), i
