"""CPU oracle of the MXFP4 mixture-of-experts operators -- TEST INFRASTRUCTURE ONLY.

Only the test suite may import this module.  It shares no code with the HIP
library and never calls it; numpy, fp64.  The pages name the experts and how
many are active per token ("When a Benchmark Crashes: The Elusive FP4 GEMM
Comparison on Blackwell SM120", section "Why This Message Was Written") and
none of these steps; the formulas are those of include/nvfp4.h.
"""
from __future__ import annotations

import numpy as np

from . import mxfp4_ref as mx
from . import nvfp4_ref as nv

SOFTMAX, SIGMOID = 0, 1
FLOOR, CEIL = 0, 1


# ---------------------------------------------------------------- routing

def scores(x: np.ndarray, score: int) -> np.ndarray:
    x = np.asarray(x, np.float64)
    with np.errstate(all="ignore"):
        if score == SIGMOID:
            return 1.0 / (1.0 + np.exp(-x))
        top = np.max(np.where(np.isnan(x), -np.inf, x), axis=-1, keepdims=True)
        p = np.exp(x - np.where(np.isneginf(top), 0.0, top))
        total = p.sum(-1, keepdims=True)
        return np.where(total == 0, 0.0, p / np.where(total == 0, 1.0, total))


def best(v: np.ndarray, n: int) -> np.ndarray:
    """Indices of the n largest of a vector, largest first, ties to the lowest index, NaN last."""
    left = [(bool(np.isnan(x)), 0.0 if np.isnan(x) else -float(x), i) for i, x in enumerate(v)]
    return np.array([i for _, _, i in sorted(left)[:n]], np.int64)


def route(logits, bias, score: int, groups: int, top_groups: int, group_top: int, top_k: int, renormalize: bool, scale):
    """(ids int32 [T][top_k], weights fp64)."""
    x = np.asarray(logits, np.float64)
    T, E = x.shape
    s = scores(x, score)
    v = s if bias is None else s + np.asarray(bias, np.float64)
    size = E // groups
    ids = np.empty((T, top_k), np.int32)
    w = np.empty((T, top_k))
    for t in range(T):
        parts = v[t].reshape(groups, size)
        sums = np.array([part[best(part, group_top)].sum() for part in parts])
        kept = sorted(best(sums, top_groups))
        experts = np.concatenate([np.arange(g * size, (g + 1) * size) for g in kept])
        ids[t] = experts[best(v[t, experts], top_k)]
        w[t] = s[t, ids[t]]
        total = w[t].sum()
        if renormalize:
            w[t] = 0.0 if total == 0 else w[t] / total
        w[t] *= np.float64(np.float32(scale))
    return ids, w


def sort_rows(ids: np.ndarray, first: int, E: int):
    """(offsets, row_token (valid rows only), token_rows), by going through the experts one by one."""
    ids = np.asarray(ids)
    token_rows = np.full(ids.shape, -1, np.int32)
    offsets, row_token = [0], []
    for e in range(first, first + E):
        for t, j in zip(*np.nonzero(ids == e)):
            token_rows[t, j] = len(row_token)
            row_token.append(t)
        offsets.append(len(row_token))
    return np.array(offsets, np.int32), np.array(row_token, np.int32), token_rows


# ----------------------------------------------------------- quantisation

def block_exponents(peak: np.ndarray, rule: int) -> np.ndarray:
    """e of blocks whose largest magnitudes are peak (finite, fp64)."""
    m, e = np.frexp(np.where(peak == 0, 1.0, peak))  # peak = m 2^e, 1/2 <= m < 1
    out = e - 3  # floor(log2 peak) - 2
    if rule == CEIL:
        out = out + (peak > 6.0 * np.exp2(out.astype(np.float64)))
    return np.clip(np.where(peak == 0, -127, out), -127, 125)


def e2m1_codes(v: np.ndarray) -> np.ndarray:
    """Nearest e2m1 codes, ties to the even code, saturating, sign kept."""
    a = np.minimum(np.abs(v), 6.0)
    grid = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
    d = np.abs(a[..., None] - grid)
    near = d == d.min(-1, keepdims=True)
    # of two equally near codes the even one
    code = np.where(near.sum(-1) == 2, np.argmax(near & (np.arange(8) % 2 == 0), -1), np.argmax(near, -1))
    return (code | (np.signbit(v).astype(np.int64) << 3)).astype(np.uint8)


def quantize(x: np.ndarray, rule: int = FLOOR):
    """(codes packed uint8 [R][K/2], scale bytes uint8 [R][K/32])."""
    x = np.asarray(x, np.float64)
    R, K = x.shape
    b = x.reshape(R, K // 32, 32)
    nan = np.isnan(b).any(-1)
    b = np.where(nan[..., None], 0.0, b)
    big = np.where(np.isinf(b), np.copysign(np.finfo(np.float32).max, b), b).astype(np.float64)
    e = block_exponents(np.abs(big).max(-1), rule)
    codes = e2m1_codes(np.where(np.isinf(b), np.copysign(6.0, b), big * np.exp2(-e.astype(np.float64))[..., None]))
    codes = np.where(nan[..., None], 0, codes).reshape(R, K)
    sf = np.where(nan, 0xFF, e + 127).astype(np.uint8)
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8), sf


# ------------------------------------------------------- grouped products

def expert_products(a, a_sf, row_token, b, b_sf, offsets, rows: int):
    """(s, mag): s[r][n] = sum_k A[row(r)] B_e and the sums of the terms'
    magnitudes, fp64 [rows][N], NaN rows where no expert covers them."""
    xa = mx.dequant(a, a_sf)
    N = b.shape[1]
    s, mag = np.full((rows, N), np.nan), np.full((rows, N), np.nan)
    for e in range(b.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            at = np.arange(lo, hi) if row_token is None else np.asarray(row_token[lo:hi])
            inside = (at >= 0) & (at < xa.shape[0])
            A = np.where(inside[:, None], xa[np.where(inside, at, 0)], 0.0)
            B = mx.dequant(b[e], b_sf[e])
            s[lo:hi], mag[lo:hi] = A @ B.T, np.abs(A) @ np.abs(B).T
    return s, mag


def activation(x: np.ndarray, act: int) -> np.ndarray:
    from math import erf, sqrt
    with np.errstate(over="ignore"):
        if act == 1:
            return np.maximum(x, 0.0)
        if act == 2:
            return 0.5 * x * (1.0 + np.vectorize(erf)(x / sqrt(2.0)))
        if act == 3:
            return 0.5 * x * (1.0 + np.tanh(np.sqrt(2.0 / np.pi) * (x + 0.044715 * x ** 3)))
        if act == 4:
            return x / (1.0 + np.exp(-x))
    return x


def moe_ffn(x, row_token, offsets, w_gu, w_gu_sf, alpha_gu, bias_gu, act, rule, w_d, w_d_sf, alpha_d, bias_d, token_rows,
            weight):
    """The layer in fp64, rounded only where its definition rounds (x and h to
    MXFP4, the down rows to bf16): out [T][H] before its own rounding."""
    rows, I = token_rows.size, w_gu.shape[1] // 2
    per_row = np.zeros(rows, np.int64)
    for e in range(w_gu.shape[0]):
        per_row[offsets[e]:offsets[e + 1]] = e
    s, _ = expert_products(*quantize(x, rule), row_token, w_gu, w_gu_sf, offsets, rows)
    s = np.nan_to_num(s)
    al = np.ones(2 * w_gu.shape[0]) if alpha_gu is None else np.asarray(alpha_gu, np.float64)
    bg = np.zeros(w_gu.shape[:2]) if bias_gu is None else np.asarray(bias_gu, np.float64)
    g = al[2 * per_row][:, None] * s[:, :I] + bg[per_row][:, :I]
    u = al[2 * per_row + 1][:, None] * s[:, I:] + bg[per_row][:, I:]
    s, _ = expert_products(*quantize(activation(g, act) * u, rule), None, w_d, w_d_sf, offsets, rows)
    s = np.nan_to_num(s)
    ad = np.ones(w_d.shape[0]) if alpha_d is None else np.asarray(alpha_d, np.float64)
    bd = np.zeros(w_d.shape[:2]) if bias_d is None else np.asarray(bias_d, np.float64)
    down = nv.bf16_to_f64(nv.bf16_rne(ad[per_row][:, None] * s + bd[per_row]))
    out = np.zeros(x.shape)
    for t in range(x.shape[0]):
        for j in range(token_rows.shape[1]):
            if token_rows[t, j] >= 0:
                out[t] += np.float64(weight[t, j]) * down[token_rows[t, j]]
    return out
