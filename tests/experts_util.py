"""Operands and comparisons of the mixture-of-experts tests."""
from __future__ import annotations

import numpy as np
import torch

import synth
from oracle import experts_ref as x
from oracle import mxfp4_ref as mx
from oracle import nvfp4_ref as nv

BF16_HALF = 2.0 ** -8   # largest relative error of a rounding to bf16
U = 2.0 ** -24          # and to fp32


def mx_operand(seed: int, *shape: int, lo: int = 122, hi: int = 130):
    """Random codes uint8 [...][K/2] and scale bytes uint8 [...][K/32] in [lo, hi]."""
    rows, K = int(np.prod(shape[:-1])), shape[-1]
    q = synth.random_codes(seed, rows, K).reshape(*shape[:-1], K // 2)
    sf = np.random.default_rng(seed + 1).integers(lo, hi + 1, (rows, K // 32)).astype(np.uint8)
    return q, sf.reshape(*shape[:-1], K // 32)


def offsets_of(counts) -> np.ndarray:
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def product_bound(s, mag, K: int, alpha=1.0, bias=0.0):
    """|bf16(fp32 alpha s + bias) - exact|: fp32 sums of K exact products in any order (K U of the
    magnitudes), a product and a sum with alpha and bias, one rounding to bf16."""
    sums = np.abs(alpha) * (K + 2) * U * mag + 2 * U * np.abs(bias)
    return BF16_HALF * (np.abs(alpha * s + bias) + sums) + sums + 2.0 ** -133


def check_mx(q, sf, h, delta, rule: int, label: str):
    """q, sf are the MXFP4 quantisation of values within delta of h: scales of a peak that near, codes
    within half a step of a value that near."""
    R, K = h.shape
    peak, slop = np.abs(h).reshape(R, -1, 32).max(-1), delta.reshape(R, -1, 32).max(-1)
    e = sf.astype(np.int64) - 127
    lo, hi = x.block_exponents(np.maximum(peak - slop, 0), rule), x.block_exponents(peak + slop, rule)
    assert ((e >= lo) & (e <= hi)).all(), f"{label}: {int(((e < lo) | (e > hi)).sum())} scales are off"
    r = np.repeat(np.exp2(-e.astype(np.float64)), 32, axis=1)
    v, d = h * r, delta * r
    code = nv.E2M1_LUT[nv.unpack_codes(q)]
    a = np.minimum(np.abs(v), 6.0)
    half = np.where(a + d < 2, 0.25, np.where(a + d < 4, 0.5, 1.0))
    off = np.abs(code - np.clip(v, -6.0, 6.0))
    assert (off <= half + d + 1e-12).all(), f"{label}: {int((off > half + d + 1e-12).sum())} codes are off"


def dev_mx(*arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in arrays]


def out_bytes(rows: int, cols: int, per: int):
    """uint8 output of rows x cols / per bytes, filled with 0xA5."""
    return torch.full((rows, cols // per), 0xA5, dtype=torch.uint8, device="cuda")
