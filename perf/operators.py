"""Measured cases of the operators around the MoE dispatch and combine: the
gate that routes tokens to experts, the residual addition with RMS norm and
8-bit output, the grouped fp8 product with 128-blocks of scales, and the fp8
expert FFN built on it.

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

def _gate(name, tokens, experts, topk, score, dtype, bias, groups, topk_groups, renormalise, scale):
    return dict(name=name, op="gate", tokens=tokens, experts=experts, topk=topk, score=score, dtype=dtype, bias=bias,
                groups=groups, topk_groups=topk_groups, renormalise=renormalise, scale=scale)


def _norm(name, rows, hidden, dtype, residual, weight, quant, y):
    return dict(name=name, op="norm", rows=rows, hidden=hidden, dtype=dtype, residual=residual, weight=weight,
                quant=quant, y=y)


def _gmm(name, rows, experts, empty, n, k):
    return dict(name=name, op="gmm", rows=rows, experts=experts, empty=empty, n=n, k=k)


def _ffn(name, rows, experts, empty, hidden, inter, quant_input):
    return dict(name=name, op="ffn", rows=rows, experts=experts, empty=empty, hidden=hidden, inter=inter,
                quant_input=quant_input)


def listed():
    return [
        # one rank's decode step: 32 tokens, 256 experts in 8 groups, biased sigmoid scores
        _gate("gate decode", 32, 256, 8, "sigmoid", "fp32", True, 8, 4, True, 2.5),
        # the share step's 8 x 2048 tokens over 128 experts, softmax scores of bf16 logits
        _gate("gate share", 16384, 128, 8, "softmax", "bf16", False, 1, 1, True, 1.0),
        # a long prefill over 256 experts in groups
        _gate("gate prefill", 32768, 256, 8, "sigmoid", "fp32", True, 8, 4, True, 2.5),
        # decode step: new residual, bf16 rows for the gate and the dispatch, fp8 rows for the shared expert
        _norm("norm decode", 32, 7168, "bf16", "bf16", "bf16", "fp8", True),
        # the share step's tokens
        _norm("norm share", 16384, 7168, "bf16", "bf16", "bf16", "fp8", True),
        # odd sizes, a residual stream kept in fp32, int8 rows for the int8 FFN
        _norm("norm int8 odd", 2051, 5000, "fp16", "fp32", "fp32", "int8", False),
        # a decode step's rows over 32 local experts (two of them get none)
        _gmm("gmm decode", 256, 32, 2, 4096, 7168),
        # one matrix (shared expert) at 2048 tokens
        _gmm("gmm dense", 2048, 1, 0, 4096, 7168),
        # ragged experts and sizes off every tile
        _gmm("gmm ragged", 3001, 7, 1, 1160, 2000),
        # expert FFN of a decode step
        _ffn("ffn decode", 256, 32, 2, 7168, 4096, False),
        # expert FFN of the share step: about 16384 rows over 16 local experts
        _ffn("ffn share", 16384, 16, 0, 7168, 4096, False),
        # shared expert on rows that the norm already quantised
        _ffn("ffn shared expert", 512, 1, 0, 7168, 4096, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gate", "norm", "gmm", "ffn"])
    if op == "gate":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * rng.randint(max(2, 16 // groups), 512 // groups)
        topk_groups = rng.randint((groups + 1) // 2, groups)
        c = _gate("", _log(rng, 1, 16384), experts, rng.randint(1, min(16, experts // groups * topk_groups)),
                  rng.choice(["softmax", "sigmoid"]), rng.choice(["bf16", "fp16", "fp32"]), rng.random() < 0.5, groups,
                  topk_groups, rng.random() < 0.7, rng.choice([1.0, 2.5]))
    elif op == "norm":
        dtype = rng.choice(["bf16", "fp16"])
        quant = rng.choice(["none", "int8", "fp8", "fp8"])
        c = _norm("", _log(rng, 1, 8192), 8 * _log(rng, 8, 1024), dtype, rng.choice(["none", dtype, dtype, "fp32"]),
                  rng.choice([dtype, "fp32"]), quant, quant == "none" or rng.random() < 0.5)
    elif op == "gmm":
        experts = _log(rng, 1, 32)
        empty = rng.randint(0, experts // 4)
        c = _gmm("", experts + _log(rng, 1, 8192), experts, empty, 8 * _log(rng, 16, 512), 16 * _log(rng, 8, 448))
    else:
        experts = _log(rng, 1, 16)
        empty = rng.randint(0, experts // 4)
        c = _ffn("", experts + _log(rng, 1, 8192), experts, empty, 128 * rng.randint(2, 56), 256 * rng.randint(1, 16),
                 rng.random() < 0.5)
    del c["name"]
    return c


def work(case):
    c = case
    if c["op"] == "gate":
        t, e = c["tokens"], c["experts"]
        # per score: an exponential, a product or two, a comparison for each of the choices
        return {"bytes": t * e * BYTES[c["dtype"]] + (4 * e if c["bias"] else 0) + t * c["topk"] * 8,
                "flops": t * e * 4}
    if c["op"] == "norm":
        t, h, b = c["rows"], c["hidden"], BYTES[c["dtype"]]
        n = t * h * b + h * BYTES[c["weight"]]
        if c["residual"] != "none":
            n += 2 * t * h * BYTES[c["residual"]]
        if c["y"]:
            n += t * h * b
        if c["quant"] != "none":
            n += t * h + 4 * t * (1 if c["quant"] == "int8" else -(-h // BLOCK))
        return {"bytes": n, "flops": 6 * t * h}
    live = c["experts"] - c["empty"]
    if c["op"] == "gmm":
        r, n, k = c["rows"], c["n"], c["k"]
        nb, kb = -(-n // BLOCK), -(-k // BLOCK)
        return {"bytes": r * (k + 4 * kb + 2 * n) + live * (n * k + 4 * nb * kb) + 8 * c["experts"],
                "flops": 2 * r * n * k}
    r, h, n = c["rows"], c["hidden"], c["inter"]
    weights = live * (n * h + h * n // 2) * (1 + 4 / BLOCK ** 2)
    return {"bytes": int(r * h * (1 + 4 / BLOCK if c["quant_input"] else 2) + r * h * 2 + weights) + 8 * c["experts"],
            "flops": 2 * r * (n * h + h * (n // 2))}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _counts(case, seed):
    """Rows of each expert: uneven, `empty` of the experts get none, the others at least one."""
    g = np.random.default_rng([seed, 17])
    live = case["experts"] - case["empty"]
    share = g.dirichlet(np.full(live, 4.0))
    some = 1 + g.multinomial(case["rows"] - live, share)
    counts = np.zeros(case["experts"], np.int64)
    counts[np.sort(g.permutation(case["experts"])[:live])] = some
    return counts.tolist()


def _fp8_weights(gen, experts, n, k):
    """Weights as a quantised checkpoint holds them: normal values whose 128 x 128 blocks reach about 448."""
    w = (torch.randn((experts, n, k), generator=gen, device=DEV, dtype=torch.bfloat16) * 100).clamp_(-448, 448)
    scale = torch.rand((experts, -(-n // BLOCK), -(-k // BLOCK)), generator=gen, device=DEV) + 0.5
    return w.to(E4M3), scale * (0.01 / math.sqrt(k))


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 11)
    s = dict(case)
    if c["op"] == "gate":
        t, e = c["tokens"], c["experts"]
        s["logits"] = (1.5 * torch.randn((t, e), generator=gen, device=DEV)).to(TYPES[c["dtype"]])
        s["bias_t"] = 0.1 * torch.randn((e,), generator=gen, device=DEV) if c["bias"] else None
        s["ids"] = torch.empty((t, c["topk"]), dtype=torch.int32, device=DEV)
        s["scales"] = torch.empty((t, c["topk"]), dtype=torch.float32, device=DEV)
        return s
    if c["op"] == "norm":
        t, h, dt = c["rows"], c["hidden"], TYPES[c["dtype"]]
        s["x"] = torch.randn((t, h), generator=gen, device=DEV).to(dt)
        # channels of a residual stream differ in size, a few by a lot
        spread = torch.exp(0.7 * torch.randn((h,), generator=gen, device=DEV))
        s["res"] = s["res_out"] = None
        if c["residual"] != "none":
            s["res"] = (3 * spread * torch.randn((t, h), generator=gen, device=DEV)).to(TYPES[c["residual"]])
            s["res_out"] = torch.empty_like(s["res"])
        s["weight_t"] = (1 + 0.2 * torch.randn((h,), generator=gen, device=DEV)).to(TYPES[c["weight"]])
        s["eps"] = 1e-6
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
    counts = _counts(c, seed)
    rows = c["rows"] + 37      # the buffers are larger than the rows in use
    s["counts"] = counts
    s["nums"] = torch.tensor(counts, dtype=torch.int64, device=DEV)
    k = c["k"] if c["op"] == "gmm" else c["hidden"]
    x = torch.randn((rows, k), generator=gen, device=DEV)
    if c["op"] == "gmm" or c["quant_input"]:
        s["a"], s["a_scale"] = _plain_quant(x)
    else:
        s["x"] = x.to(torch.bfloat16)
    if c["op"] == "gmm":
        s["w"], s["w_scale"] = _fp8_weights(gen, c["experts"], c["n"], k)
        s["y_t"] = torch.zeros((rows, c["n"]), dtype=torch.bfloat16, device=DEV)
        return s
    s["w1"], s["w1_scale"] = _fp8_weights(gen, c["experts"], c["inter"], k)
    s["w2"], s["w2_scale"] = _fp8_weights(gen, c["experts"], k, c["inter"] // 2)
    s["y_t"] = torch.zeros((rows, k), dtype=torch.bfloat16, device=DEV)
    if own:   # the workspace that the framework's size query asks for, which a program keeps between calls
        import combine_route_histogram_amd as mdc
        s["shape"] = mdc.Shape(1, 0, rows, k, 1, c["experts"], rows)
        s["workspace"] = torch.empty(mdc.mdc_ffn_fp8_workspace(s["shape"], c["inter"]), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_gate(s):
    z = s["logits"].double()
    off = torch.isnan(z) | (z == -math.inf)
    z = torch.where(off, torch.full_like(z, -math.inf), z)
    if s["score"] == "softmax":
        top = z.amax(1, keepdim=True)
        p = torch.exp(z - torch.where(top == -math.inf, torch.zeros_like(top), top))
        total = p.sum(1, keepdim=True)
        p = p / torch.where(total > 0, total, torch.ones_like(total))
    else:
        p = 1 / (1 + torch.exp(-z))
    t, e, g, k = s["tokens"], s["experts"], s["groups"], s["topk"]
    # without a bias the order is that of the logits
    key = z if s["bias_t"] is None and g == 1 else p + (0 if s["bias_t"] is None else s["bias_t"].double())
    key = torch.where(off, torch.full_like(key, -math.inf), key)
    if g > 1:
        per = key.view(t, g, e // g)
        best = torch.sort(per, dim=2, descending=True).values[:, :, :2 if s["bias_t"] is not None else 1].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :s["topk_groups"]]
        open_ = torch.zeros((t, g), dtype=torch.bool, device=z.device).scatter_(1, kept, True)
        key = torch.where(open_[:, :, None], per, torch.full_like(per, -math.inf)).reshape(t, e)
    order = torch.sort(key, dim=1, descending=True, stable=True)
    ids, none = order.indices[:, :k], order.values[:, :k] == -math.inf
    w = torch.where(none, torch.zeros_like(p[:, :k]), torch.gather(p, 1, ids))
    if s["renormalise"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones_like(total))
    return {"ids": torch.where(none, torch.full_like(ids, -1), ids).to(torch.int32),
            "scales": (w * s["scale"]).float()}


def _plain_quant(v):
    """fp32 rows -> e4m3 codes and one scale for each 128 columns."""
    rows, h = v.shape
    nb = -(-h // BLOCK)
    p = torch.nn.functional.pad(v, (0, nb * BLOCK - h)).view(rows, nb, BLOCK)
    amax = p.abs().amax(2)
    amax = torch.where(amax > 0, amax.clamp_min(AMAX_MIN), amax)
    # 448 v is exact for 16-bit v, so halves between two codes stay halves
    codes = (FP8_MAX * p / torch.where(amax > 0, amax, torch.ones_like(amax))[:, :, None]).clamp(-FP8_MAX, FP8_MAX)
    return codes.view(rows, nb * BLOCK)[:, :h].contiguous().to(E4M3), amax / FP8_MAX


def _plain_norm(s):
    v = s["x"].float()
    out = {}
    if s["res"] is not None:
        v = v + s["res"].float()
        out["residual"] = v.to(s["res"].dtype)
    inv = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + s["eps"])
    v = v * inv * s["weight_t"].float()
    if s["y_t"] is not None:
        out["y"] = v.to(s["y_t"].dtype)
    if s["quant"] == "fp8":
        out["q"], out["q_scale"] = _plain_quant(v)
    elif s["quant"] == "int8":
        amax = v.abs().amax(1)
        codes = torch.round(v * torch.where(amax > 0, 127 / amax, torch.zeros_like(amax))[:, None]).clamp(-127, 127)
        out["q_scale"] = amax / 127
        out["q"] = (codes * out["q_scale"][:, None]).to(torch.bfloat16)
    return out


def _plain_values(codes, scale):
    """fp8 rows as the fp32 values they stand for."""
    return codes.float() * scale.repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]


def _plain_product(a, a_scale, w, w_scale, counts):
    """Rows of each expert times that expert's transposed weights, in fp32."""
    n = w.shape[1]
    used = _plain_values(a, a_scale)[:sum(counts)].split(counts)
    return torch.cat([rows @ _plain_values(w[e], w_scale[e].repeat_interleave(BLOCK, 0)[:n]).t()
                      for e, rows in enumerate(used)])


def _plain_ffn(s):
    a, a_scale = (s["a"], s["a_scale"]) if s["quant_input"] else _plain_quant(s["x"].float())
    h = _plain_product(a, a_scale, s["w1"], s["w1_scale"], s["counts"])
    gate, up = h.chunk(2, 1)
    q, q_scale = _plain_quant(gate / (1 + torch.exp(-gate)) * up)
    return {"y": _plain_product(q, q_scale, s["w2"], s["w2_scale"], s["counts"]).to(torch.bfloat16)}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    s = state
    if own:
        return _own(s)
    if s["op"] == "gate":
        return _plain_gate(s)
    if s["op"] == "norm":
        return _plain_norm(s)
    if s["op"] == "gmm":
        return {"y": _plain_product(s["a"], s["a_scale"], s["w"], s["w_scale"], s["counts"]).to(torch.bfloat16)}
    return _plain_ffn(s)


def _own(s):
    import combine_route_histogram_amd as mdc
    if s["op"] == "gate":
        shape = mdc.Shape(1, 0, s["tokens"], 8, s["topk"], s["experts"], 0)
        mdc.mdc_gate(shape, s["logits"], s["bias_t"], s["ids"], s["scales"], score=s["score"], groups=s["groups"],
                     topk_groups=s["topk_groups"], group_top=2 if s["groups"] > 1 and s["bias"] else 1,
                     renormalise=s["renormalise"], scale=s["scale"])
        return {"ids": s["ids"], "scales": s["scales"]}
    if s["op"] == "norm":
        mdc.mdc_add_rms_norm(s["x"], s["weight_t"], residual=s["res"], residual_out=s["res_out"], y=s["y_t"],
                             q=s["q"], q_scale=s["q_scale"], eps=s["eps"])
        out = {}
        if s["res"] is not None:
            out["residual"] = s["res_out"]
        if s["y_t"] is not None:
            out["y"] = s["y_t"]
        if s["quant"] != "none":
            out["q_scale"] = s["q_scale"]
            # int8 codes as the values they stand for
            out["q"] = torch.mul(s["q"], s["q_scale"][:, None], out=s["q_values"]) if s["quant"] == "int8" else s["q"]
        return out
    used = s["rows"]
    if s["op"] == "gmm":
        mdc.mdc_gmm_fp8(s["a"], s["a_scale"], s["nums"], s["w"], s["w_scale"], s["y_t"])
    elif s["quant_input"]:
        mdc.mdc_ffn_fp8_quant_input(s["shape"], s["inter"], s["a"], s["a_scale"], s["nums"], s["w1"], s["w1_scale"],
                                    s["w2"], s["w2_scale"], s["y_t"], s["workspace"])
    else:
        mdc.mdc_ffn_fp8(s["shape"], s["inter"], s["x"], s["nums"], s["w1"], s["w1_scale"], s["w2"], s["w2_scale"],
                        s["y_t"], s["workspace"])
    return {"y": s["y_t"][:used]}


# ---------------------------------------------------------------------------
# 64 bits
# ---------------------------------------------------------------------------

def _exact_gate(s):
    z = s["logits"].double().cpu().numpy()
    live = np.isfinite(z)
    z = np.where(live, z, -np.inf)
    if s["score"] == "softmax":
        p = np.exp(z - z.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
    else:
        p = 1.0 / (1.0 + np.exp(-z))
    t, e, g, k = s["tokens"], s["experts"], s["groups"], s["topk"]
    bias = None if s["bias_t"] is None else s["bias_t"].double().cpu().numpy()
    key = z if bias is None and g == 1 else np.where(live, p + (0.0 if bias is None else bias), -np.inf)
    if g > 1:
        size = e // g
        per = np.sort(key.reshape(t, g, size), axis=2)
        score = per[:, :, -1] + (per[:, :, -2] if bias is not None else 0.0)
        rank = np.argsort(np.argsort(-score, axis=1, kind="stable"), axis=1)
        key = np.where(np.repeat(rank < s["topk_groups"], size, axis=1), key, -np.inf)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(p, ids, 1)
    if s["renormalise"]:
        w = w / w.sum(1, keepdims=True)
    return {"ids": ids.astype(np.int32), "scales": w * s["scale"]}


def _exact_e4m3(v):
    """Nearest e4m3 value (ties to even): steps of 2^(exponent - 3), of 2^-9 below 2^-6."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-FP8_MAX, FP8_MAX)


def _exact_blocks(v):
    """64-bit rows -> (e4m3 values, scale of each 128 columns)."""
    h = v.shape[1]
    parts = v.split(BLOCK, dim=1)
    amax = torch.stack([p.abs().amax(1) for p in parts], 1)
    amax = torch.where(amax > 0, amax.clamp_min(AMAX_MIN), amax)
    wide = torch.cat([amax[:, i:i + 1].expand(-1, p.shape[1]) for i, p in enumerate(parts)], 1)
    assert wide.shape[1] == h
    codes = _exact_e4m3(v * FP8_MAX / torch.where(wide > 0, wide, torch.ones_like(wide)))
    return codes, amax / FP8_MAX


def _exact_product(values, w, w_scale, counts):
    out, at = [], 0
    for e, count in enumerate(counts):
        if count:
            n, k = w[e].shape
            cols = torch.arange(k, device=w.device) // BLOCK
            lines = torch.arange(n, device=w.device) // BLOCK
            we = w[e].double() * w_scale[e].double()[lines][:, cols]
            out.append(torch.matmul(values[at:at + count], we.t().contiguous()))
        at += count
    return torch.cat(out)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "gate":
        return _exact_gate(s)
    if s["op"] == "norm":
        v = s["x"].double()
        out = {}
        if s["res"] is not None:
            v = v + s["res"].double()
            out["residual"] = v
        v = v / torch.sqrt(v.square().mean(1, keepdim=True) + s["eps"]) * s["weight_t"].double()
        if s["y_t"] is not None:
            out["y"] = v
        if s["quant"] == "fp8":
            out["q"], out["q_scale"] = _exact_blocks(v)
        elif s["quant"] == "int8":
            scale = v.abs().amax(1) / 127
            out["q_scale"] = scale
            wide = torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]
            out["q"] = torch.round(v / wide).clamp(-127, 127) * scale[:, None]
        return out
    used = sum(s["counts"])
    if s["op"] == "gmm" or s["quant_input"]:
        cols = torch.arange(s["a"].shape[1], device=DEV) // BLOCK
        values = s["a"][:used].double() * s["a_scale"][:used].double()[:, cols]
    else:
        codes, scale = _exact_blocks(s["x"][:used].double())
        values = codes * scale[:, torch.arange(codes.shape[1], device=DEV) // BLOCK]
    if s["op"] == "gmm":
        return {"y": _exact_product(values, s["w"], s["w_scale"], s["counts"])}
    h = _exact_product(values, s["w1"], s["w1_scale"], s["counts"])
    half = h.shape[1] // 2
    codes, scale = _exact_blocks(torch.sigmoid(h[:, :half]) * h[:, :half] * h[:, half:])
    values = codes * scale[:, torch.arange(half, device=DEV) // BLOCK]
    return {"y": _exact_product(values, s["w2"], s["w2_scale"], s["counts"])}
