"""CPU oracle for the dense transformer block around the NVFP4 GEMM -- TEST
INFRASTRUCTURE ONLY.

Epilogues (bias, activation, residual), the gated feed-forward and the norms
before and after a block, in numpy from their formulas.  Only the test suite
imports this module; it shares nothing with the HIP library and never calls
it.  The pages do not describe these steps; the formulas are the usual ones.

GEMM sums are fp64 here and fp32 in the kernels, so each result comes with the
bound that the kernel's roundings allow, term by term (u = 2^-24):

* a sum s of K products: 8 sqrt(K) u ||terms||_2, the probabilistic bound of
  fp32 summation that ``nvfp4_ref.gemm_tolerance`` uses;
* alpha s, + bias, * beta, + residual, the gated product: u of the value each;
* an activation: its slope (at most 1.13) times the error of its argument, plus
  its own evaluation error, at most (16 + 4 E) u of the value, where E is the
  size of the exponential's argument (|x| for SiLU, 2 sqrt(2 / pi) (|x| +
  0.044715 |x|^3) for the tanh form, x^2 / 2 for the erf form): an argument
  made of at most 4 roundings is off by 4 E u, which the exponential turns into
  a relative error of its value; 16 u cover the polynomial of the erf form (its
  fit and 9 steps), exp2 and reciprocal (2 u each) and the remaining products;
* the output: half a bf16 step, 2^-8 of the value at most.

The norm's arithmetic is fixed step by step (fp64 sums, fp32 elsewhere), so
``residual_norm`` gives its bits.
"""
from __future__ import annotations

import math

import numpy as np

from oracle import nvfp4_ref as o

ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = range(5)
RMS, LAYER = 0, 1
U = 2.0 ** -24
_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def activation(x: np.ndarray, act: int) -> np.ndarray:
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if act == ACT_RELU:
            return np.where(x < 0, 0.0, x)
        if act == ACT_GELU:
            return 0.5 * x * _erfc(-x / math.sqrt(2.0))
        if act == ACT_GELU_TANH:
            z = math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3)
            return x / (1.0 + np.exp(-2.0 * z))
        if act == ACT_SILU:
            return x / (1.0 + np.exp(-x))
        return x


def _act_error(x, y, act, dx):
    """Bound of the fp32 activation's error for an argument off by dx."""
    if act in (ACT_NONE, ACT_RELU):
        return dx
    a = np.abs(x)
    e = {ACT_SILU: a, ACT_GELU: a * a / 2, ACT_GELU_TANH: 1.6 * a + 0.0714 * a ** 3}[act]
    return 1.13 * dx + (16.0 + 4.0 * e) * U * np.abs(y) + 2.0 ** -126


def _sum_and_error(xa, xb, alpha, bias):
    """alpha xa xb^T + bias (fp64) and the bound of its fp32 evaluation."""
    s = xa @ xb.T
    norm = np.sqrt((xa * xa) @ (xb * xb).T)
    v = np.float64(alpha) * s
    err = 8.0 * math.sqrt(xa.shape[1]) * U * norm * abs(float(alpha)) + U * np.abs(v)
    if bias is not None:
        v = v + bias[None, :]
        err = err + U * np.abs(v)
    return v, err


def epilogue(xa, xb, alpha, bias, act, residual, beta):
    """(value, bound) of act(alpha xa xb^T + bias) + beta residual before the
    bf16 rounding; xa, xb: dequantised fp64, bias and residual fp64 or None."""
    x, dx = _sum_and_error(xa, xb, alpha, bias)
    y = activation(x, act)
    err = _act_error(x, y, act, dx)
    if residual is not None:
        t = float(np.float32(beta)) * residual
        y = y + t
        err = err + U * (np.abs(t) + np.abs(y))
    return y, err


def gated(xa, xg, xu, alpha, bias, act):
    """(value, bound) of act(alpha[0] xa xg^T + bias_g) * (alpha[1] xa xu^T + bias_u)."""
    n = xg.shape[0]
    g, dg = _sum_and_error(xa, xg, alpha[0], None if bias is None else bias[:n])
    u, du = _sum_and_error(xa, xu, alpha[1], None if bias is None else bias[n:])
    a = activation(g, act)
    da = _act_error(g, a, act, dg)
    h = a * u
    return h, np.abs(u) * da + np.abs(a) * du + da * du + U * np.abs(h)


def bf16_bound(y, err):
    """Bound of the bf16 result against the unrounded value y."""
    return err + 2.0 ** -8 * (np.abs(y) + err) + 2.0 ** -133


def quantized_range(h, err, gs):
    """(lowest, highest) admissible scale bytes of every block of h +- err, by
    the quantiser's rule (monotone in the block's largest magnitude)."""
    rows, n = h.shape
    mag = np.abs(h).reshape(rows, n // 16, 16)
    e = err.reshape(rows, n // 16, 16)
    lo = np.max(np.maximum(mag - e, 0.0), axis=2)
    hi = np.max(mag + e, axis=2)
    f = lambda a: o.e4m3_encode(((a / 6.0) * float(np.float32(gs))).astype(np.float32))
    return f(lo * (1.0 - 4 * U)), f(hi * (1.0 + 4 * U))


def check_quantized(q, sf, h, err, gs, label=""):
    """The codes and scales are those of some h within err: each scale in the
    range its block allows, each code in the range that the scale found allows."""
    rows, n = h.shape
    lo, hi = quantized_range(h, err, gs)
    assert ((sf >= lo) & (sf <= hi)).all(), f"{label}: scale outside {int(((sf < lo) | (sf > hi)).sum())} ranges"
    sv = o.E4M3_LUT[sf].astype(np.float64)
    r = np.zeros_like(sv)
    r[sv != 0] = float(np.float32(gs)) / sv[sv != 0]
    r = np.repeat(r, 16, axis=1)
    wide = err + 4 * U * np.abs(h)
    at = lambda x: o.E2M1_LUT[o.e2m1_encode((x * r).astype(np.float32))].astype(np.float64)
    codes = o.E2M1_LUT[o.unpack_codes(q)].astype(np.float64)
    low, high = at(h - wide), at(h + wide)
    bad = (codes < low) | (codes > high)
    assert not bad.any(), f"{label}: {int(bad.sum())} of {bad.size} codes outside their range"


def _normed(v32, w, b, kind, eps):
    d = v32.astype(np.float64)
    mean = np.zeros((len(d), 1))
    if kind == LAYER:
        mean = d.sum(axis=1, keepdims=True) / d.shape[1]
    c = d - mean
    rstd = (1.0 / np.sqrt((c * c).sum(axis=1, keepdims=True) / d.shape[1] + np.float64(np.float32(eps)))).astype(np.float32)
    y = (c.astype(np.float32) if kind == LAYER else v32) * rstd
    if w is not None:
        y = y * w.astype(np.float32)[None, :]
    if b is not None:
        y = y + b.astype(np.float32)[None, :]
    return y


def residual_norm(x, post_w, post_b, gate, gate_group, res, beta, w, b, eps, kind):
    """fp32 r and y of the norms around a block, step by step (fp64 sums and
    rstd, fp32 elsewhere, in the formulas' order).  x, res: fp32 [T][H];
    vectors fp32; gate [rows][H]."""
    v = np.asarray(x, dtype=np.float32)
    if post_w is not None:
        v = _normed(v, post_w, post_b, kind, eps)
    if gate is not None:
        rows = np.arange(len(v)) // gate_group if gate_group > 0 else np.zeros(len(v), dtype=np.int64)
        v = gate.astype(np.float32)[rows] * v
    if res is not None:
        v = np.float32(beta) * res.astype(np.float32) + v
    return v, _normed(v, w, b, kind, eps)


def residual_norm_exact(x, post_w, post_b, gate, gate_group, res, beta, w, b, eps, kind):
    """The formulas in fp64."""
    def norm(v, w, b):
        m = v.mean(axis=1, keepdims=True) if kind == LAYER else 0.0
        y = (v - m) / np.sqrt(((v - m) ** 2).mean(axis=1, keepdims=True) + eps)
        y = y if w is None else y * w.astype(np.float64)[None, :]
        return y if b is None else y + b.astype(np.float64)[None, :]
    v = np.asarray(x, dtype=np.float64)
    if post_w is not None:
        v = norm(v, post_w, post_b)
    if gate is not None:
        rows = np.arange(len(v)) // gate_group if gate_group > 0 else np.zeros(len(v), dtype=np.int64)
        v = gate.astype(np.float64)[rows] * v
    if res is not None:
        v = float(beta) * res.astype(np.float64) + v
    return v, norm(v, w, b)
