"""Operands and comparisons of the block-operator tests."""
from __future__ import annotations

import numpy as np
import torch

import synth
from oracle import nvfp4_ref as o
from tests.gpu_util import dev


def bf16(x: np.ndarray) -> np.ndarray:
    """fp32 values -> the nearest bf16 values, as fp32."""
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).float().numpy()


def dev_bf16(x: np.ndarray) -> torch.Tensor:
    """GPU bf16 tensor of values that are bf16 already."""
    return dev(np.asarray(x, np.float32)).to(torch.bfloat16)


def values(t: torch.Tensor) -> np.ndarray:
    """A GPU bf16 tensor's values in fp64."""
    torch.cuda.synchronize()
    return t.float().cpu().numpy().astype(np.float64)


def operand(seed: int, rows: int, K: int, lo: int = 0x30, hi: int = 0x40):
    """Random codes and scale bytes and their values."""
    q = synth.random_codes(seed, rows, K)
    sf = synth.random_scale_bytes(seed + 1, rows, K, lo=lo, hi=hi)
    return q, sf, o.dequant(q, sf)


def close(got: np.ndarray, want: np.ndarray, bound: np.ndarray, label: str) -> None:
    err = np.abs(got - want)
    assert got.shape == want.shape
    assert np.isfinite(got).all(), f"{label}: not finite"
    bad = err > bound
    assert not bad.any(), (f"{label}: {int(bad.sum())} of {bad.size} outside the bound, worst {np.max(err / bound):.3g} "
                           f"times it")
