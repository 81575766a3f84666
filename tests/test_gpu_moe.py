"""mdc_moe and mdc_moe_fp8 against the 64-bit oracle, element by element.

The tokens are such that the first product is exact (int8: always; fp8: codes and scales whose products and sums fp32 holds),
so that g is off by the rounding of fp32's operations only and its codes are known but for those whose value lies that near a
border: these enter the tolerance with the step that they may be off by."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_route_histogram_amd as mdc  # noqa: E402
from oracle import ops64 as O  # noqa: E402
from tests.test_gpu_fp8 import BF, DEV, E4M3, GROUP, HALF, group_max, np64  # noqa: E402

F32 = torch.float32


def weights(fmt, g, L, n, k, lo, hi):
    if fmt == "int8":
        return (torch.randint(-127, 128, (L, n, k), generator=g, dtype=torch.int8),
                (torch.rand((L, n), generator=g) + 0.5) / (70 * k ** 0.5))
    return (torch.randint(-2, 3, (L, n, k), generator=g).to(E4M3),
            torch.exp2(torch.randint(lo, hi + 1, (L, -(-n // 128), -(-k // 128)), generator=g).float()))


def widen(fmt, w, s):
    return np64(w) * np64(s)[:, :, None] if fmt == "int8" else O.fp8_widen(np64(w.float()), np64(s))


def tokens(fmt, g, T, H):
    if fmt == "int8":
        return torch.randn((T, H), generator=g).to(BF)
    # 448 and 224 times a power of two in each run of 128: the codes are 448 and 224 (or 448 alone), the scale a power of two
    size = torch.exp2(torch.randint(-10, -7, (T, H // 128, 1), generator=g).float())
    return (224.0 * torch.randint(-2, 3, (T, H // 128, 128), generator=g) * size).view(T, H).to(BF)


class Layer:
    def __init__(self, fmt, T, K, H, N, E, world=1, rank=0, zero=0, copy=0, seed=0, mask=None):
        g = self.g = torch.Generator().manual_seed(seed)
        self.fmt, self.T, self.K, self.H, self.N = fmt, T, K, H, N
        self.L = E // world
        self.shape = mdc.Shape(world, rank, T, H, K, E, 0, zero_experts=zero, copy_experts=copy,
                               mask_per_route=int(mask == "route"))
        self.x = tokens(fmt, g, T, H)
        self.w1, self.s1 = weights(fmt, g, self.L, N, H, -5, -4)
        self.w2, self.s2 = weights(fmt, g, self.L, H, N // 2, -4, -1)
        self.n = E + zero + copy
        self.ids = torch.stack([torch.randperm(self.n, generator=g)[:K] for _ in range(T)]).to(torch.int32) if T else \
            torch.zeros((0, K), dtype=torch.int32)
        self.scales = torch.softmax(torch.randn((T, K), generator=g), 1) * 2
        self.mask = None if mask is None else torch.rand((T, K) if mask == "route" else (T,), generator=g) < 0.7
        self.shared = torch.randn((T, H), generator=g).to(BF)
        self.logits = None
        self.gate = {}

    def run(self, shared=True, ori=True, guard=2, **over):
        d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        self.out = torch.full((self.T + guard, self.H), 3.0, dtype=BF, device=DEV)
        call, size = (mdc.mdc_moe, mdc.mdc_moe_workspace) if self.fmt == "int8" else \
            (mdc.mdc_moe_fp8, mdc.mdc_moe_fp8_workspace)
        self.ws = torch.full((size(self.shape, self.N) + 256,), 0x5A, dtype=torch.uint8, device=DEV)
        if self.logits is not None:
            self.got_ids = torch.full((self.T, self.K), -7, dtype=torch.int32, device=DEV)
            self.got_scales = torch.full((self.T, self.K), -7.0, device=DEV)
        else:
            self.got_ids, self.got_scales = d(self.ids), d(self.scales)
        args = dict(x=d(self.x), logits=d(self.logits), bias=None, expert_ids=self.got_ids,
                    expert_scales=self.got_scales, w1=d(self.w1), w1_scale=d(self.s1), w2=d(self.w2), w2_scale=d(self.s2),
                    x_out=self.out, workspace=self.ws[:-256], x_active_mask=d(self.mask),
                    shared_expert_x=d(self.shared) if shared else None, ori_x=d(self.x) if ori else None)
        args.update(self.gate)
        args.update(over)
        call(self.shape, self.N, **args)
        torch.cuda.synchronize()
        assert (self.out[self.T:] == 3).all() and (self.ws[-256:] == 0x5A).all()
        return self.out[:self.T].cpu()

    def check(self, shared=True, ori=True, sharp=True):
        got = np64(self.run(shared, ori))
        sh, fmt, I = self.shape, self.fmt, self.N // 2
        ids, scales = self.got_ids.cpu().numpy(), np64(self.got_scales)
        mask = None if self.mask is None else self.mask.numpy()
        weight, has, cp, present, dropped = O.moe_routes(ids, scales, mask, sh.rank * self.L, self.L, sh.num_experts,
                                                         sh.zero_experts, sh.copy_experts)
        assert mdc.read_status(self.ws) == {"dropped_ids": dropped, "overflow_rows": 0, "wait_timeouts": 0}
        x = np64(self.x)
        want, size, tol = np.zeros((self.T, self.H)), np.zeros((self.T, self.H)), np.zeros((self.T, self.H))
        if fmt == "int8":   # codes as fp32 decides them
            x32 = self.x.float().numpy()
            amax = np.abs(x32).max(1, initial=0)
            inv = np.where(amax > 0, np.float32(127) / np.where(amax > 0, amax, 1).astype(np.float32), 0).astype(np.float32)
            values = np.clip(np.rint(x32 * inv[:, None]), -127, 127).astype(np.float64) * amax[:, None] / 127
        else:
            values = O.fp8_widen(*O.fp8_quant(x))
            assert np.array_equal(values, x)
        depth = 2.0 ** -23 * (8 + has.sum() * (I // 128) + 16)   # additions to an output's sum
        for e in range(self.L):
            rows = np.flatnonzero(has[:, e])
            if rows.size == 0:
                continue
            h = values[rows] @ widen(fmt, self.w1[e:e + 1], self.s1[e:e + 1])[0].T
            gate, up = h[:, :I], h[:, I:]
            v = gate / (1 + np.exp(-gate)) * up
            # h (int8: its conversion, amax / 127 and two products): 4 roundings, which the exponential takes times |gate|;
            # silu: the exponential's argument times 1 / ln 2 (two roundings), the exponential and the reciprocal of 2^-23
            # each, the sum and two products
            rel = ((2 + 4) * np.abs(gate).max() + 2 + 2 + 3 + 8) * 2.0 ** -24
            if fmt == "int8":
                codes, s = O.int8_quant(v)
                wide = np.repeat(s[:, None], I, 1)
                rounded = lambda u: np.clip(np.rint(u), -127, 127)  # noqa: E731
            else:
                codes, s = O.fp8_quant(v)
                wide = O.fp8_widen(np.ones_like(v), s)
                rounded = lambda u: O.e4m3_round(np.clip(u, -448, 448))  # noqa: E731
            value = v / np.where(wide > 0, wide, 1)
            off = (2 * rel + 8 * 2.0 ** -24) * np.abs(value)   # of v and of the amax
            unsure = np.maximum(np.abs(rounded(value + off) - codes), np.abs(rounded(value - off) - codes)) * wide
            w2 = widen(fmt, self.w2[e:e + 1], self.s2[e:e + 1])[0]
            v2, wt = codes * wide, weight[rows, e][:, None]
            want[rows] += wt * (v2 @ w2.T)
            part = np.abs(v2) @ np.abs(w2).T
            size[rows] += np.abs(wt) * part
            tol[rows] += np.abs(wt) * (unsure @ np.abs(w2).T + (rel + 8 * 2.0 ** -24) * part)
            if fmt == "fp8":
                tol[rows] += np.abs(wt) * GROUP * O.grouped(group_max(v2), group_max(w2[None]), [rows.size])
        if ori:
            want += cp[:, None] * x
            size += np.abs(cp[:, None] * x)
        if shared:
            want += present[:, None] * np64(self.shared)
            size += np.abs(present[:, None] * np64(self.shared))
        tol += HALF * np.abs(want) + (depth + 20 * 2.0 ** -24) * size
        err = np.abs(got - want)
        assert np.all(err <= tol), (err / np.maximum(tol, 1e-30)).max()
        if sharp and has.any() and not shared:   # an error of 5% in an element is past the bound for most of them
            assert np.mean(0.05 * np.abs(want) > tol) > 0.5
        return got


FMT = pytest.mark.parametrize("fmt", ["int8", "fp8"])


@FMT
@pytest.mark.parametrize("T", [1, 2, 7, 15, 16, 17, 31, 32])
def test_tokens(fmt, T):
    Layer(fmt, T, 3, 512, 512, 12, seed=T).check(shared=False)


@FMT
@pytest.mark.parametrize("H", [128, 256, 384, 1024, 1152, 2048, 2560, 4096, 7168, 8192])
def test_hidden_sizes(fmt, H):
    Layer(fmt, 5, 2, H, 512, 4, seed=H).check(shared=False)
    Layer(fmt, 18, 2, H, 256, 2, seed=H + 1).check()


@FMT
@pytest.mark.parametrize("N", [256, 512, 768, 1280, 4096, 8192])
def test_inner_sizes(fmt, N):
    Layer(fmt, 4, 2, 256, N, 5, seed=N).check(shared=False)
    Layer(fmt, 32, 1, 128, N, 1, seed=N + 1).check()   # all tokens on one expert


@FMT
@pytest.mark.parametrize("K,E", [(1, 1), (1, 64), (8, 8), (8, 256), (16, 16), (16, 40)])
def test_routes(fmt, K, E):
    for T in (1, 9, 32):
        Layer(fmt, T, K, 256, 256, E, seed=K + E + T).check()


@FMT
def test_many_experts(fmt):
    Layer(fmt, 32, 16, 128, 256, 2048, seed=3).check()


@FMT
def test_ranks_give_parts_of_one_sum(fmt):
    """The parts of all ranks, each against the oracle; ids of other ranks' experts are no part of it."""
    for rank in range(4):
        Layer(fmt, 12, 4, 256, 512, 16, world=4, rank=rank, seed=5).check(shared=rank == 1)
    Layer(fmt, 3, 1, 256, 512, 64, world=32, rank=31, seed=6).check(sharp=False)


@FMT
@pytest.mark.parametrize("mask", [None, "token", "route"])
@pytest.mark.parametrize("zero,copy", [(0, 0), (3, 0), (0, 3), (4, 5)])
def test_zero_and_copy_experts_and_masks(fmt, mask, zero, copy):
    m = Layer(fmt, 20, 5, 384, 512, 6, zero=zero, copy=copy, mask=mask, seed=zero + 10 * copy)
    got = m.check()
    if mask == "token":
        assert not got[~m.mask.numpy()].any()   # a token that is off gets zeros


@FMT
def test_ids_that_repeat_or_are_out_of_range(fmt):
    m = Layer(fmt, 6, 6, 256, 512, 8, seed=7)
    m.ids[0] = torch.tensor([3, 3, 3, 1, 1, 3])
    m.ids[1] = torch.tensor([8, -1, 7, 100, -2 ** 31, 2 ** 31 - 1])
    m.ids[2] = -1
    m.ids[3] = 5
    got = m.check(shared=False)
    assert not got[2].any()


@FMT
def test_no_route_at_all(fmt):
    m = Layer(fmt, 4, 2, 256, 512, 8, seed=8)
    m.ids[:] = -1
    assert not m.check(shared=True).any()
    m = Layer(fmt, 4, 2, 256, 512, 8, world=2, rank=1, seed=8)
    m.ids[:] = 1   # all on the other rank
    m.check(shared=True)


@FMT
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF, torch.float16, F32])
@pytest.mark.parametrize("T", [1, 8, 9, 32])
def test_with_its_gate(fmt, score, dtype, T):
    m = Layer(fmt, T, 4, 256, 512, 32, zero=4, copy=4, seed=T)
    m.logits = (1.5 * torch.randn((T, 40), generator=m.g)).to(dtype)
    bias = 0.1 * torch.randn(40, generator=m.g) if score == "sigmoid" else None
    m.gate = dict(score=score, bias=None if bias is None else bias.to(DEV), groups=4, topk_groups=2, group_top=2, scale=1.5)
    m.check()
    ids, w = O.gate(np64(m.logits), None if bias is None else bias.numpy(), 4, score, 4, 2, 2, True, 1.5)
    assert np.array_equal(ids, m.got_ids.cpu().numpy())
    want_i, want_w = torch.empty_like(m.got_ids), torch.empty_like(m.got_scales)
    one = mdc.Shape(1, 0, T, 256, 4, 32, 0, zero_experts=4, copy_experts=4)
    mdc.mdc_gate(one, m.logits.to(DEV), m.gate["bias"], want_i, want_w, score=score, groups=4, topk_groups=2, group_top=2,
                 scale=1.5)
    assert torch.equal(want_i, m.got_ids) and torch.equal(want_w, m.got_scales)


@FMT
@pytest.mark.parametrize("T,n", [(1, 8), (3, 65), (8, 129), (2, 513), (1, 1040), (5, 2048)])
def test_gates_of_many_experts(fmt, T, n):
    m = Layer(fmt, T, 4, 128, 256, n, seed=n)
    m.logits = torch.randn((T, n), generator=m.g)
    m.logits[0, 1] = m.logits[0].max()      # a tie, ids that are off
    m.logits[0, 0] = float("nan")
    m.logits[T - 1, 2:n // 2] = float("-inf")
    m.check()
    ids, _ = O.gate(np64(m.logits), None, 4)
    assert np.array_equal(ids, m.got_ids.cpu().numpy())


@FMT
def test_the_gates_routes_may_stay_inside(fmt):
    m = Layer(fmt, 6, 4, 256, 512, 32, seed=11)
    m.logits = torch.randn((6, 32), generator=m.g)
    a = m.run()
    b = m.run(expert_ids=None, expert_scales=None)
    assert torch.equal(a, b)


@FMT
def test_fewer_ids_on_than_choices(fmt):
    m = Layer(fmt, 3, 4, 256, 512, 8, seed=12)
    m.logits = torch.randn((3, 8), generator=m.g)
    m.logits[1, 2:] = float("-inf")
    m.logits[2] = float("-inf")
    got = m.check(shared=False)
    assert not got[2].any()


@FMT
def test_what_is_not_finite_reaches_its_tokens_only(fmt):
    """NaN in a token's row, in an expert's scales, an infinite route scale."""
    m = Layer(fmt, 20, 2, 256, 512, 8, seed=13)
    m.ids[:] = torch.tensor([0, 1])
    m.ids[4] = torch.tensor([2, 3])
    m.ids[9] = torch.tensor([4, 5])
    m.ids[18] = torch.tensor([1, 6])
    clean = m.run()
    m.x[4, 17] = float("nan")
    m.s2[5] = float("nan")
    m.s1[6] = float("inf")
    m.scales[0, 1] = float("inf")
    got = m.run(ori=False)
    bad = ~torch.isfinite(got.float()).all(1)
    assert bad.nonzero().flatten().tolist() == [0, 4, 9, 18]
    keep = [t for t in range(20) if t not in (0, 4, 9, 18)]
    assert torch.equal(got[keep], clean[keep])


@FMT
def test_what_is_not_finite_where_no_route_looks(fmt):
    """The rows of masked tokens, the copy row of a token without a copy expert, the scales of masked and dropped routes."""
    m = Layer(fmt, 18, 2, 256, 512, 8, copy=2, seed=17)
    m.ids[:] = torch.tensor([0, 1])
    m.ids[2] = torch.tensor([3, 9])    # one copy expert
    m.ids[5] = torch.tensor([-1, 10])   # no present route
    m.mask = torch.ones(18, dtype=torch.bool)
    m.mask[[1, 17]] = False
    ori = m.x.clone()
    clean = m.run(ori_x=ori.to(DEV))
    for t in (1, 17):
        m.x[t, 3], m.shared[t, 7], m.scales[t, 0] = float("nan"), float("inf"), float("nan")
    m.shared[5], m.scales[5] = float("nan"), float("inf")
    ori[[0, 1, 3, 5, 17]] = float("nan")
    got = m.run(ori_x=ori.to(DEV))
    assert torch.equal(got, clean) and not got[[1, 5, 17]].any()
    assert torch.isfinite(got.float()).all()


@FMT
def test_zero_rows_and_rows_of_other_sizes(fmt):
    m = Layer(fmt, 6, 2, 256, 512, 4, seed=14)
    m.x[1] = 0
    m.x[2] *= 2.0 ** -40
    m.x[3, :128] = 0
    m.check(shared=False, sharp=False)


@FMT
def test_x_out_may_be_an_input(fmt):
    m = Layer(fmt, 6, 3, 256, 512, 4, copy=3, seed=15)
    want = m.run(guard=0)
    for name in ("x", "shared_expert_x"):
        t = (m.x if name == "x" else m.shared).to(DEV)
        over = {name: t, "x_out": t}
        if name == "x":
            over["ori_x"] = t
        m.run(guard=0, **over)
        assert torch.equal(t.cpu(), want), name


@FMT
@pytest.mark.parametrize("gated", [False, True])
def test_streams_graphs_and_repeats(fmt, gated):
    T, K, H, N, E = 13, 4, 512, 768, 24
    m = Layer(fmt, T, K, H, N, E, seed=16)
    if gated:
        m.logits = torch.randn((T, E), generator=m.g)
    first = m.run(guard=0)
    for _ in range(3):
        assert torch.equal(m.run(guard=0), first)
    d = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    prep, size = (mdc.prepare_moe, mdc.mdc_moe_workspace) if fmt == "int8" else (mdc.prepare_moe_fp8,
                                                                                  mdc.mdc_moe_fp8_workspace)
    x, ids, sc, lg, shared = d(m.x), d(m.ids), d(m.scales), d(m.logits), d(m.shared)
    fixed = [d(t) for t in (m.w1, m.s1, m.w2, m.s2)]

    def bound(stream=None):
        out = torch.zeros((T, H), dtype=BF, device=DEV)
        ws = torch.empty(size(m.shape, N), dtype=torch.uint8, device=DEV)
        r = (torch.empty_like(ids), torch.empty_like(sc)) if gated else (ids, sc)
        return prep(m.shape, N, x, lg, None, *r, *fixed, out, ws, shared_expert_x=shared, stream=stream), out

    call, a = bound()
    call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other, b = bound()
        other()
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a.cpu(), first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured, c = bound()
        captured()
    for rep in range(4):
        x.copy_(torch.randn((T, H), device=DEV).to(BF))
        ids.copy_(torch.randint(-1, E, (T, K), device=DEV, dtype=torch.int32))
        if gated:
            lg.copy_(torch.randn((T, E), device=DEV))
        c.zero_()
        graph.replay()
        call()
        torch.cuda.synchronize()
        assert torch.equal(a, c) and a.any(), rep


@FMT
def test_no_tokens(fmt):
    m = Layer(fmt, 0, 2, 256, 512, 4, seed=17)
    m.run()
    assert (m.ws == 0x5A).all()


@FMT
def test_it_follows_the_chain_of_calls(fmt):
    """gate, dispatch, expert FFN and combine give the same but for the roundings of y (and, int8, g) to 16 bits that the
    chain makes: half a step of bf16 for each, relative to sums that cancel by no more than the bound counts."""
    T, K, H, N, E = 24, 4, 512, 1024, 16
    g = torch.Generator().manual_seed(18)
    x = torch.randn((T, H), generator=g).to(BF).to(DEV)
    logits = torch.randn((T, E), generator=g).to(DEV)
    shared = torch.randn((T, H), generator=g).to(BF).to(DEV)
    w1, s1 = (t.to(DEV) for t in weights(fmt, g, E, N, H, -5, -4))
    w2, s2 = (t.to(DEV) for t in weights(fmt, g, E, H, N // 2, -4, -1))
    if fmt == "fp8":
        s1, s2 = s1 / 4, s2 / 16
    A = T * K
    sh = mdc.Shape(1, 0, T, H, K, E, A)
    ids, sc = torch.empty((1, T, K), dtype=torch.int32, device=DEV), torch.empty((1, T, K), device=DEV)
    mdc.mdc_gate(sh, logits, None, ids, sc)
    o = mdc.alloc_dispatch_outputs(sh)
    idx = torch.full((1, T, K), -1, dtype=torch.int32, device=DEV)
    mdc.mdc_dispatch(sh, x, ids, None, o["expand_x"], o["assist_info"], o["ep_recv_counts"], o["expert_token_nums"], idx,
                     o["workspace"])
    y = torch.empty((A, H), dtype=BF, device=DEV)
    ffn, size = (mdc.mdc_ffn, mdc.mdc_ffn_workspace) if fmt == "int8" else (mdc.mdc_ffn_fp8, mdc.mdc_ffn_fp8_workspace)
    ws = torch.empty(size(sh, N), dtype=torch.uint8, device=DEV)
    ffn(sh, N, o["expand_x"], o["expert_token_nums"], w1, s1, w2, s2, y, ws)
    chain = torch.empty((T, H), dtype=BF, device=DEV)
    mdc.mdc_combine(sh, [y], [o["assist_info"]], [o["ep_recv_counts"]], idx, ids, sc, None, shared, chain)
    out = torch.empty((T, H), dtype=BF, device=DEV)
    call, size = (mdc.mdc_moe, mdc.mdc_moe_workspace) if fmt == "int8" else (mdc.mdc_moe_fp8, mdc.mdc_moe_fp8_workspace)
    ws2 = torch.empty(size(sh, N), dtype=torch.uint8, device=DEV)
    call(sh, N, x, logits, None, None, None, w1, s1, w2, s2, out, ws2, shared_expert_x=shared)
    a, b = chain.double(), out.double()
    # bf16 of y and of the sum 2^-8 each at most; int8: g's bf16 rounding may move a code by one, a step of amax / 127 in
    # some of N / 2 terms of random sign
    rel = ((a - b).norm() / a.norm()).item()
    assert rel < (2 * 2.0 ** -8 if fmt == "fp8" else 2 * 2.0 ** -8 + 1 / 127), rel
