"""The gate, the residual RMS norm, the fp8 block quantiser, the grouped fp8
product and the fp8 expert FFN in 64 bits, from their definitions (numpy on the
CPU; shares nothing with the HIP path)."""
from __future__ import annotations

import numpy as np

BLOCK = 128
FP8_MAX = 448.0
AMAX_MIN = 2.0 ** -110


# ---- e4m3 ----

def e4m3_values() -> np.ndarray:
    """Value of each of the 256 codes (OCP e4m3: bias 7, no infinities, S.1111.111 is NaN)."""
    out = np.empty(256)
    for c in range(256):
        sign, e, m = -1.0 if c & 0x80 else 1.0, (c >> 3) & 15, c & 7
        if e == 15 and m == 7:
            out[c] = np.nan
        else:
            out[c] = sign * (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return out


def e4m3_round(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value of |v| <= 448, ties to even."""
    _, e = np.frexp(np.abs(v))
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.clip(np.rint(v / step) * step, -FP8_MAX, FP8_MAX)


def fp8_quant(v: np.ndarray):
    """[rows][H] -> (values of the codes, scales [rows][ceil(H/128)])."""
    rows, h = v.shape
    nb = -(-h // BLOCK)
    codes, scales = np.empty_like(v), np.empty((rows, nb))
    for b in range(nb):
        part = v[:, b * BLOCK:(b + 1) * BLOCK]
        amax = np.abs(part).max(1)
        a = np.where(amax > 0, np.maximum(amax, AMAX_MIN), 1.0)
        codes[:, b * BLOCK:(b + 1) * BLOCK] = e4m3_round(part * FP8_MAX / a[:, None])
        scales[:, b] = np.where(amax > 0, a / FP8_MAX, 0.0)
    return codes, scales


def fp8_widen(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """codes [..., rows, H], scales [..., rows or blocks of rows, ceil(H/128)] -> the values they stand for."""
    cols = np.arange(codes.shape[-1]) // BLOCK
    if scales.shape[-2] != codes.shape[-2]:
        scales = scales[..., np.arange(codes.shape[-2]) // BLOCK, :]
    return codes * scales[..., cols]


# ---- gate ----

def gate(logits, bias, topk, score="softmax", groups=1, topk_groups=1, group_top=1, renormalise=True, scale=1.0):
    """-> (ids [T][K], weights [T][K]); id -1, weight 0 where fewer than K ids are on."""
    z = np.asarray(logits, np.float64).copy()
    z[np.isnan(z)] = -np.inf
    z = np.minimum(z, np.finfo(np.float32).max)
    T, n = z.shape
    ids = np.full((T, topk), -1, np.int32)
    weights = np.zeros((T, topk))
    for t in range(T):
        on = z[t] > -np.inf
        p = np.zeros(n)
        if score == "softmax":
            if on.any():
                p[on] = np.exp(z[t][on] - z[t][on].max())
                p /= p.sum()
        else:
            p[on] = 1 / (1 + np.exp(-z[t][on]))
        key = z[t].copy() if bias is None and groups == 1 else p + (0 if bias is None else np.asarray(bias, float))
        key[~on | np.isnan(key)] = -np.inf
        if groups > 1:
            size = n // groups
            best = [np.sort(key[g * size:(g + 1) * size])[::-1][:group_top].sum() for g in range(groups)]
            order = sorted(range(groups), key=lambda g: (-best[g], g))
            for g in order[topk_groups:]:
                key[g * size:(g + 1) * size] = -np.inf
        order = sorted(range(n), key=lambda e: (-key[e], e))[:topk]
        got = [e for e in order if key[e] > -np.inf]
        ids[t, :len(got)] = got
        w = p[got]
        if renormalise and w.sum() > 0:
            w = w / w.sum()
        weights[t, :len(got)] = w * scale
    return ids, weights


# ---- norm ----

def add_rms_norm(x, residual, weight, eps):
    """-> (h, v) in 64 bits: the sum, and the normalised row before any rounding."""
    h = np.asarray(x, np.float64) + (0 if residual is None else np.asarray(residual, np.float64))
    return h, h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * np.asarray(weight, np.float64)


# ---- products ----

def grouped(a, w, counts):
    """Rows of a by expert (counts), each times its expert's w [L][n][K] transposed."""
    out, at = [], 0
    for e, c in enumerate(counts):
        out.append(a[at:at + c] @ w[e].T)
        at += c
    return np.concatenate(out)


def ffn_fp8(q1, w1, w2, counts):
    """q1, w1, w2: values (codes times scales).  -> y in 64 bits (the rounding of g to fp8 is part of the formula)."""
    h = grouped(q1, w1, counts)
    half = h.shape[1] // 2
    gate_, up = h[:, :half], h[:, half:]
    return grouped(fp8_widen(*fp8_quant(gate_ / (1 + np.exp(-gate_)) * up)), w2, counts)
