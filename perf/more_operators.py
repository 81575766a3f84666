"""Measured cases of the operators that serve a layer in 8 bits: the grouped
int8 product with scales for each token and channel, the norms before and after
a block with its gate and residual scale, and a whole mixture-of-experts layer
for a few tokens with int8 or fp8 experts.

`run` computes an operator in plain torch, or through the package where `own`
is true; `exact` gives the same outputs from the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
BLOCK = 128                 # elements of a row (rows x columns of a weight) that share one fp8 scale
FP8_MAX = 448.0             # largest e4m3 value
AMAX_MIN = 2.0 ** -110      # a non-zero block's amax is taken as at least this, so that 1 / amax is finite
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _gmm(name, rows, experts, empty, n, k, dtype):
    return dict(name=name, op="gmm", rows=rows, experts=experts, empty=empty, n=n, k=k, dtype=dtype)


def _norm(name, rows, hidden, dtype, post, residual, weight, gate, act, every, quant, y):
    """gate: none, row (one value a row), channel (a row of them for all rows), sequence (for `every` rows), element."""
    return dict(name=name, op="norm", rows=rows, hidden=hidden, dtype=dtype, post=post, residual=residual,
                weight=weight, gate=gate, act=act, every=every, quant=quant, y=y)


def _moe(name, fmt, tokens, world, experts, zero, copy, topk, hidden, inter, gate, score, dtype, bias, groups,
         topk_groups, shared):
    """gate false: the routes are given."""
    return dict(name=name, op="moe", fmt=fmt, tokens=tokens, world=world, experts=experts, zero=zero, copy=copy,
                topk=topk, hidden=hidden, inter=inter, gate=gate, score=score, dtype=dtype, bias=bias, groups=groups,
                topk_groups=topk_groups, shared=shared)


def listed():
    return [
        # one token through one matrix (the shared expert's second product in decode)
        _gmm("gmm one token", 1, 1, 0, 7168, 2048, "bf16"),
        # a decode step's rows over 32 local experts (two of them get none)
        _gmm("gmm decode", 256, 32, 2, 4096, 7168, "bf16"),
        # one matrix at a prefill's 4096 tokens
        _gmm("gmm dense", 4096, 1, 0, 4096, 7168, "bf16"),
        # ragged experts and sizes off every tile
        _gmm("gmm ragged", 3001, 7, 1, 1160, 2000, "fp16"),
        # decode step: a learned scale for each channel of the block's output, 16-bit rows for the gate, fp8 rows for
        # the shared expert
        _norm("block norm decode", 32, 7168, "bf16", True, "bf16", "bf16", "channel", "none", 1, "fp8", True),
        # the share step's 8 x 2048 tokens, a gate row for each sequence
        _norm("block norm share", 16384, 7168, "bf16", True, "bf16", "bf16", "sequence", "none", 2048, "fp8", True),
        # odd sizes, a residual stream kept in fp32, a sigmoid gate for each element, int8 rows for the int8 experts
        _norm("block norm int8 odd", 2051, 5000, "fp16", True, "fp32", "fp32", "element", "sigmoid", 1, "int8", False),
        # one token of a chat through a layer of 32 experts
        _moe("moe one token", "fp8", 1, 1, 32, 0, 0, 8, 7168, 4096, True, "softmax", "bf16", False, 1, 1, False),
        # one rank's share of a decode step: 32 tokens, 32 of 256 experts, biased sigmoid scores in groups
        _moe("moe decode", "fp8", 32, 8, 256, 0, 0, 8, 7168, 4096, True, "sigmoid", "fp32", True, 8, 4, True),
        # a layer of many small experts at a handful of tokens, zero and copy experts among the ids
        _moe("moe small experts", "int8", 5, 1, 128, 8, 8, 8, 2048, 1536, True, "softmax", "fp32", False, 1, 1, True),
        # int8 experts of the share step's size on routes that were made elsewhere
        _moe("moe int8", "int8", 16, 8, 128, 0, 0, 8, 7168, 4096, False, "softmax", "fp32", False, 1, 1, False),
        # the smallest call: one token, small experts
        _moe("moe small one token", "int8", 1, 1, 64, 0, 0, 4, 1024, 1024, True, "softmax", "bf16", False, 1, 1, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gmm", "norm", "moe"])
    if op == "gmm":
        experts = _log(rng, 1, 32)
        empty = rng.randint(0, experts // 4)
        c = _gmm("", experts - empty + _log(rng, 1, 4096) - 1, experts, empty, 8 * _log(rng, 16, 512),
                 16 * _log(rng, 8, 448), rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    elif op == "norm":
        dtype = rng.choice(["bf16", "fp16"])
        quant = rng.choice(["none", "int8", "fp8", "fp8"])
        gate = rng.choice(["none", "row", "channel", "sequence", "element"])
        rows = _log(rng, 1, 8192)
        c = _norm("", rows, 8 * _log(rng, 8, 1024), dtype, rng.random() < 0.8, rng.choice(["none", dtype, dtype, "fp32"]),
                  rng.choice([dtype, "fp32"]), gate, rng.choice(["none", "sigmoid", "tanh"]) if gate != "none" else "none",
                  rng.randint(1, rows) if gate == "sequence" else 1, quant, quant == "none" or rng.random() < 0.5)
    else:
        world = rng.choice([1, 1, 2, 4, 8])
        groups = rng.choice([1, 1, 2, 4])
        local = groups * _log(rng, 1, 32 // groups)
        experts = local * world
        zero, copy = (rng.choice([0, 4, 8]), rng.choice([0, 4, 8])) if groups == 1 else (0, 0)
        ids = experts + zero + copy
        topk_groups = rng.randint((groups + 1) // 2, groups)
        gate = rng.random() < 0.7
        c = _moe("", rng.choice(["int8", "fp8"]), _log(rng, 1, 32), world, experts, zero, copy,
                 rng.randint(1, min(8, ids // groups * topk_groups)), 128 * _log(rng, 2, 56), 256 * _log(rng, 1, 16),
                 gate, rng.choice(["softmax", "sigmoid"]), rng.choice(["bf16", "fp16", "fp32"]), rng.random() < 0.5,
                 groups, topk_groups, rng.random() < 0.5)
    del c["name"]
    return c


def work(case):
    c = case
    if c["op"] == "gmm":
        r, n, k, live = c["rows"], c["n"], c["k"], c["experts"] - c["empty"]
        return {"bytes": r * (k + 4 + n * BYTES[c["dtype"]]) + live * n * (k + 4) + 8 * c["experts"],
                "flops": 2 * r * n * k}
    if c["op"] == "norm":
        t, h, b = c["rows"], c["hidden"], BYTES[c["dtype"]]
        n = t * h * b + h * BYTES[c["weight"]] * (2 if c["post"] else 1)
        n += t * h * BYTES[c["residual"] if c["residual"] != "none" else c["dtype"]] * (2 if c["residual"] != "none" else 1)
        n += {"none": 0, "row": t, "channel": h, "sequence": -(-t // c["every"]) * h, "element": t * h}[c["gate"]] * b
        if c["y"]:
            n += t * h * b
        if c["quant"] != "none":
            n += t * h + 4 * t * (1 if c["quant"] == "int8" else -(-h // BLOCK))
        return {"bytes": n, "flops": 12 * t * h}
    t, h, n, e = c["tokens"], c["hidden"], c["inter"], c["experts"]
    ids, local = e + c["zero"] + c["copy"], e // c["world"]
    # experts that get a token, and routes, as they are to be expected of even routing
    hit = local * (1 - (1 - c["topk"] / ids) ** t)
    routes = t * c["topk"] * local / ids
    scales = 4 / BLOCK ** 2 if c["fmt"] == "fp8" else 0
    expert = (n * h + h * n // 2) * (1 + scales) + (4 * (n + h) if c["fmt"] == "int8" else 0)
    rows = t * h * 2 * (2 + c["shared"]) + t * c["topk"] * 8 + (t * ids * BYTES[c["dtype"]] if c["gate"] else 0)
    return {"bytes": int(hit * expert + rows), "flops": int(2 * routes * (n * h + h * (n // 2)))}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _counts(case, seed):
    """Rows of each expert: uneven, `empty` of the experts get none, the others at least one."""
    g = np.random.default_rng([seed, 23])
    live = case["experts"] - case["empty"]
    some = 1 + g.multinomial(case["rows"] - live, g.dirichlet(np.full(live, 4.0)))
    counts = np.zeros(case["experts"], np.int64)
    counts[np.sort(g.permutation(case["experts"])[:live])] = some
    return counts.tolist()


def _int8_weights(gen, experts, n, k):
    """Weights as a quantised checkpoint holds them: codes over the whole range, a scale for each output channel."""
    w = torch.randint(-127, 128, (experts, n, k), generator=gen, device=DEV, dtype=torch.int8)
    scale = torch.rand((experts, n), generator=gen, device=DEV) + 0.5
    return w, scale * (1 / (73 * math.sqrt(k)))


def _fp8_weights(gen, experts, n, k):
    """Normal values whose 128 x 128 blocks reach about 448, and a scale for each block."""
    w = (torch.randn((experts, n, k), generator=gen, device=DEV, dtype=torch.bfloat16) * 100).clamp_(-448, 448)
    scale = torch.rand((experts, -(-n // BLOCK), -(-k // BLOCK)), generator=gen, device=DEV) + 0.5
    return w.to(E4M3), scale * (0.01 / math.sqrt(k))


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(int(seed) * 6007 + 29)
    randn = lambda *shape: torch.randn(shape, generator=gen, device=DEV)  # noqa: E731
    s = dict(case)
    if c["op"] == "gmm":
        rows = c["rows"] + 37      # the buffers are larger than the rows in use
        s["counts"] = _counts(c, seed)
        s["nums"] = torch.tensor(s["counts"], dtype=torch.int64, device=DEV)
        s["a"], s["a_scale"] = _plain_int8(randn(rows, c["k"]))
        s["w"], s["w_scale"] = _int8_weights(gen, c["experts"], c["n"], c["k"])
        s["y_t"] = torch.zeros((rows, c["n"]), dtype=TYPES[c["dtype"]], device=DEV)
        return s
    if c["op"] == "norm":
        t, h, dt = c["rows"], c["hidden"], TYPES[c["dtype"]]
        # channels of a residual stream differ in size, a few by a lot
        spread = torch.exp(0.7 * randn(h))
        s["x"] = (2 * randn(t, h)).to(dt)
        s["res"] = (3 * spread * randn(t, h)).to(TYPES[c["residual"]]) if c["residual"] != "none" else None
        s["res_out"] = torch.empty((t, h), dtype=dt if s["res"] is None else s["res"].dtype, device=DEV)
        s["post_t"] = (1 + 0.2 * randn(h)).to(TYPES[c["weight"]]) if c["post"] else None
        s["weight_t"] = (1 + 0.2 * randn(h)).to(TYPES[c["weight"]])
        shape = {"none": None, "row": (t, 1), "channel": (1, h), "sequence": (-(-t // c["every"]), h), "element": (t, h)}
        s["gate_t"] = None if c["gate"] == "none" else (0.5 + 0.3 * randn(*shape[c["gate"]])).to(dt)
        s["gate_every"] = {"channel": max(t, 1), "sequence": c["every"]}.get(c["gate"], 1)
        s["block_scale"], s["residual_scale"], s["eps"] = 0.75, 1.25, 1e-6
        s["y_t"] = torch.empty((t, h), dtype=dt, device=DEV) if c["y"] else None
        s["q"] = s["q_scale"] = None
        if c["quant"] == "int8":
            s["q"] = torch.empty((t, h), dtype=torch.int8, device=DEV)
            s["q_scale"] = torch.empty((t,), dtype=torch.float32, device=DEV)
            s["q_values"] = torch.empty((t, h), dtype=torch.bfloat16, device=DEV)
        elif c["quant"] == "fp8":
            s["q"] = torch.empty((t, h), dtype=E4M3, device=DEV)
            s["q_scale"] = torch.empty((t, -(-h // BLOCK)), dtype=torch.float32, device=DEV)
        return s
    t, h, n, k = c["tokens"], c["hidden"], c["inter"], c["topk"]
    ids, local = c["experts"] + c["zero"] + c["copy"], c["experts"] // c["world"]
    weights = _int8_weights if c["fmt"] == "int8" else _fp8_weights
    s["x"] = randn(t, h).to(torch.bfloat16)
    s["w1"], s["w1_scale"] = weights(gen, local, n, h)
    s["w2"], s["w2_scale"] = weights(gen, local, h, n // 2)
    s["shared_t"] = randn(t, h).to(torch.bfloat16) if c["shared"] else None
    s["rank"] = c["world"] // 2
    s["logits"] = s["bias_t"] = None
    if c["gate"]:
        s["logits"] = (1.5 * randn(t, ids)).to(TYPES[c["dtype"]])
        s["bias_t"] = 0.1 * randn(ids) if c["bias"] else None
        s["ids"] = torch.empty((t, k), dtype=torch.int32, device=DEV)
        s["scales"] = torch.empty((t, k), dtype=torch.float32, device=DEV)
    else:
        s["ids"] = torch.argsort(randn(t, ids), dim=1)[:, :k].to(torch.int32).contiguous()
        s["scales"] = torch.softmax(randn(t, k), dim=1)
    s["out"] = torch.empty((t, h), dtype=torch.bfloat16, device=DEV)
    if own:   # the workspace that the framework's size query asks for, which a program keeps between calls
        import combine_route_histogram_amd as mdc
        s["shape"] = mdc.Shape(c["world"], s["rank"], t, h, k, c["experts"], 0, zero_experts=c["zero"],
                               copy_experts=c["copy"])
        size = mdc.mdc_moe_workspace if c["fmt"] == "int8" else mdc.mdc_moe_fp8_workspace
        s["workspace"] = torch.empty(size(s["shape"], n), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_int8(v):
    """fp32 rows -> int8 codes and a scale for each row."""
    amax = v.abs().amax(1)
    codes = torch.round(v * torch.where(amax > 0, 127 / amax, torch.zeros_like(amax))[:, None]).clamp(-127, 127)
    return codes.to(torch.int8), amax / 127


def _plain_fp8(v):
    """fp32 rows -> e4m3 codes and one scale for each 128 columns."""
    rows, h = v.shape
    nb = -(-h // BLOCK)
    p = torch.nn.functional.pad(v, (0, nb * BLOCK - h)).view(rows, nb, BLOCK)
    amax = p.abs().amax(2)
    amax = torch.where(amax > 0, amax.clamp_min(AMAX_MIN), amax)
    codes = (FP8_MAX * p / torch.where(amax > 0, amax, torch.ones_like(amax))[:, :, None]).clamp(-FP8_MAX, FP8_MAX)
    return codes.view(rows, nb * BLOCK)[:, :h].contiguous().to(E4M3), amax / FP8_MAX


def _plain_gmm(s):
    counts = s["counts"]
    rows = s["a"][:sum(counts)].float().split(counts)
    acc = torch.cat([r @ s["w"][e].float().t() * s["w_scale"][e] for e, r in enumerate(rows)])
    return {"y": (acc * s["a_scale"][:sum(counts), None]).to(s["y_t"].dtype)}


def _plain_rms(v, weight, eps):
    return v / torch.sqrt((v * v).mean(1, keepdim=True) + eps) * weight.float()


def _plain_norm(s):
    v = s["x"].float()
    if s["post_t"] is not None:
        v = _plain_rms(v, s["post_t"], s["eps"])
    v = v * s["block_scale"]
    if s["gate_t"] is not None:
        g = s["gate_t"].float()
        if s["act"] == "sigmoid":
            g = 1 / (1 + torch.exp(-g))
        elif s["act"] == "tanh":
            g = torch.tanh(g)
        v = v * g.repeat_interleave(s["gate_every"], 0)[:v.shape[0]]
    if s["res"] is not None:
        v = v + s["residual_scale"] * s["res"].float()
    out = {"residual": v.to(s["res_out"].dtype)}
    v = _plain_rms(v, s["weight_t"], s["eps"])
    if s["y_t"] is not None:
        out["y"] = v.to(s["y_t"].dtype)
    if s["quant"] == "fp8":
        out["q"], out["q_scale"] = _plain_fp8(v)
    elif s["quant"] == "int8":
        q, out["q_scale"] = _plain_int8(v)
        out["q"] = (q.float() * out["q_scale"][:, None]).to(torch.bfloat16)
    return out


def _plain_gate(s):
    """Ids and weights; the choice is made in 64 bits (keys next to each other)."""
    z = s["logits"].double()
    if s["score"] == "softmax":
        p = torch.exp(z - z.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-z))
    t, n = z.shape
    g = s["groups"]
    key = z if s["bias_t"] is None and g == 1 else p + (0 if s["bias_t"] is None else s["bias_t"].double())
    if g > 1:
        per = key.view(t, g, n // g)
        best = torch.sort(per, dim=2, descending=True).values[:, :, :_group_top(s)].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        open_ = torch.zeros((t, g), dtype=torch.bool, device=z.device).scatter_(1, kept, True)
        key = torch.where(open_[:, :, None], per, torch.full_like(per, -math.inf)).reshape(t, n)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :s["topk"]]
    w = torch.gather(p, 1, ids)
    return ids.to(torch.int32), (w / w.sum(1, keepdim=True)).float()


def _group_top(s):
    """Keys of a group that make its score."""
    return 2 if s["bias_t"] is not None and (s["experts"] + s["zero"] + s["copy"]) // s["groups"] > 1 else 1


def _plain_moe(s):
    ids, scales = _plain_gate(s) if s["gate"] else (s["ids"], s["scales"])
    local = s["experts"] // s["world"]
    x = s["x"].float()
    int8 = s["fmt"] == "int8"

    def product(rows, w, w_scale):   # the rows in 8 bits, times one expert's weights
        if int8:
            q, scale = _plain_int8(rows)
            return q.float() @ w.float().t() * scale[:, None] * w_scale
        q, scale = _plain_fp8(rows)
        wide = w_scale.repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)
        return (q.float() * scale.repeat_interleave(BLOCK, 1)) @ (w.float() * wide).t()

    out = torch.zeros_like(x)
    for e in range(local):
        weight = torch.where(ids == s["rank"] * local + e, scales, torch.zeros_like(scales)).sum(1, keepdim=True)
        gate, up = product(x, s["w1"][e], s["w1_scale"][e]).chunk(2, 1)
        out = out + weight * product(gate / (1 + torch.exp(-gate)) * up, s["w2"][e], s["w2_scale"][e])
    if s["copy"]:
        out = out + torch.where(ids >= s["experts"] + s["zero"], scales, torch.zeros_like(scales)).sum(1, keepdim=True) * x
    if s["shared_t"] is not None:
        out = out + scales.sum(1, keepdim=True) * s["shared_t"].float()
    out = {"out": out.to(torch.bfloat16)}
    if s["gate"]:
        out["ids"], out["scales"] = ids, scales
    return out


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    s = state
    if own:
        return _own(s)
    return {"gmm": _plain_gmm, "norm": _plain_norm, "moe": _plain_moe}[s["op"]](s)


def _own(s):
    import combine_route_histogram_amd as mdc
    if s["op"] == "gmm":
        mdc.mdc_gmm_int8(s["a"], s["a_scale"], s["nums"], s["w"], s["w_scale"], s["y_t"])
        return {"y": s["y_t"][:s["rows"]]}
    if s["op"] == "norm":
        mdc.mdc_block_rms_norm(s["x"], s["weight_t"], post_weight=s["post_t"], gate=s["gate_t"],
                               gate_every=s["gate_every"], gate_act=s["act"], residual=s["res"],
                               residual_out=s["res_out"], y=s["y_t"], q=s["q"], q_scale=s["q_scale"],
                               block_scale=s["block_scale"], residual_scale=s["residual_scale"], post_eps=s["eps"],
                               eps=s["eps"])
        out = {"residual": s["res_out"]}
        if s["y_t"] is not None:
            out["y"] = s["y_t"]
        if s["quant"] != "none":
            out["q_scale"] = s["q_scale"]
            # int8 codes as the values they stand for
            out["q"] = torch.mul(s["q"], s["q_scale"][:, None], out=s["q_values"]) if s["quant"] == "int8" else s["q"]
        return out
    call = mdc.mdc_moe if s["fmt"] == "int8" else mdc.mdc_moe_fp8
    call(s["shape"], s["inter"], s["x"], s["logits"], s["bias_t"], s["ids"], s["scales"], s["w1"], s["w1_scale"],
         s["w2"], s["w2_scale"], s["out"], s["workspace"], shared_expert_x=s["shared_t"],
         ori_x=s["x"] if s["copy"] else None, score=s["score"], groups=s["groups"], topk_groups=s["topk_groups"],
         group_top=_group_top(s))
    out = {"out": s["out"]}
    if s["gate"]:
        out["ids"], out["scales"] = s["ids"], s["scales"]
    return out


# ---------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------

def _exact_gate(s):
    z = s["logits"].double().cpu().numpy()
    if s["score"] == "softmax":
        p = np.exp(z - z.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
    else:
        p = 1.0 / (1.0 + np.exp(-z))
    t, n = z.shape
    g = s["groups"]
    bias = None if s["bias_t"] is None else s["bias_t"].double().cpu().numpy()
    key = z if bias is None and g == 1 else p + (0.0 if bias is None else bias)
    if g > 1:
        per = np.sort(key.reshape(t, g, n // g), axis=2)
        score = per[:, :, -_group_top(s):].sum(2)
        rank = np.argsort(np.argsort(-score, axis=1, kind="stable"), axis=1)
        key = np.where(np.repeat(rank < s["topk_groups"], n // g, axis=1), key, -np.inf)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :s["topk"]]
    w = np.take_along_axis(p, ids, 1)
    return ids.astype(np.int32), w / w.sum(1, keepdims=True)


def _exact_e4m3(v):
    """Nearest e4m3 value (ties to even): steps of 2^(exponent - 3), of 2^-9 below 2^-6."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-FP8_MAX, FP8_MAX)


def _exact_blocks(v):
    """64-bit rows -> (e4m3 values, scale of each 128 columns)."""
    parts = v.split(BLOCK, dim=1)
    amax = torch.stack([p.abs().amax(1) for p in parts], 1)
    amax = torch.where(amax > 0, amax.clamp_min(AMAX_MIN), amax)
    wide = torch.cat([amax[:, i:i + 1].expand(-1, p.shape[1]) for i, p in enumerate(parts)], 1)
    codes = _exact_e4m3(v * FP8_MAX / torch.where(wide > 0, wide, torch.ones_like(wide)))
    return codes, amax / FP8_MAX


def _exact_rows(v):
    """64-bit rows -> (int8 codes as numbers, scale of each row)."""
    scale = v.abs().amax(1) / 127
    return torch.round(v / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]).clamp(-127, 127), scale


def _exact_moe(s):
    if s["gate"]:
        ids, weights = _exact_gate(s)
    else:
        ids, weights = s["ids"].cpu().numpy(), s["scales"].double().cpu().numpy()
    local = s["experts"] // s["world"]
    x = s["x"].double()
    out = torch.zeros_like(x)
    int8 = s["fmt"] == "int8"
    for e in range(local):
        mine = ids == s["rank"] * local + e
        rows = np.flatnonzero(mine.any(1))
        if rows.size == 0:
            continue
        at = torch.from_numpy(rows).to(DEV)
        v = x[at]
        for w, scale in ((s["w1"], s["w1_scale"]), (s["w2"], s["w2_scale"])):
            w, scale = w[e].double(), scale[e].double()
            if int8:
                q, row = _exact_rows(v)
                h = torch.matmul(q, w.t().contiguous()) * row[:, None] * scale[None, :]
            else:
                q, row = _exact_blocks(v)
                cols = torch.arange(w.shape[1], device=DEV) // BLOCK
                w = w * scale[torch.arange(w.shape[0], device=DEV) // BLOCK][:, cols]
                h = torch.matmul(q * row[:, cols], w.t().contiguous())
            half = h.shape[1] // 2
            v = torch.sigmoid(h[:, :half]) * h[:, :half] * h[:, half:]
        factor = torch.from_numpy((weights * mine).sum(1)[rows]).to(DEV)
        out[at] += factor[:, None] * h
    if s["copy"]:
        out += torch.from_numpy((weights * (ids >= s["experts"] + s["zero"])).sum(1)).to(DEV)[:, None] * x
    if s["shared_t"] is not None:
        out += torch.from_numpy(weights.sum(1)).to(DEV)[:, None] * s["shared_t"].double()
    return {"out": out, "ids": ids, "scales": weights} if s["gate"] else {"out": out}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "gmm":
        at, ys = 0, []
        for e, count in enumerate(s["counts"]):
            if count:
                y = torch.matmul(s["a"][at:at + count].double(), s["w"][e].double().t().contiguous())
                ys.append(y * s["a_scale"][at:at + count, None].double() * s["w_scale"][e].double())
            at += count
        return {"y": torch.cat(ys)}
    if s["op"] == "moe":
        return _exact_moe(s)
    u = s["x"].double()
    if s["post_t"] is not None:
        u = u / torch.sqrt(u.square().mean(1, keepdim=True) + s["eps"]) * s["post_t"].double()
    if s["gate_t"] is not None:
        g = s["gate_t"].double()
        g = torch.sigmoid(g) if s["act"] == "sigmoid" else torch.tanh(g) if s["act"] == "tanh" else g
        rows = torch.arange(u.shape[0], device=DEV) // s["gate_every"]
        u = u * g[rows]
    u = s["block_scale"] * u
    if s["res"] is not None:
        u = u + s["residual_scale"] * s["res"].double()
    out = {"residual": u}
    v = u / torch.sqrt(u.square().mean(1, keepdim=True) + s["eps"]) * s["weight_t"].double()
    if s["y_t"] is not None:
        out["y"] = v
    if s["quant"] == "fp8":
        out["q"], out["q_scale"] = _exact_blocks(v)
    elif s["quant"] == "int8":
        codes, out["q_scale"] = _exact_rows(v)
        out["q"] = codes * out["q_scale"][:, None]
    return out
