"""MXFP4 quantisation against the oracle, bit for bit, and with the product that
reads it."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_07_amd as nv
from oracle import experts_ref as x
from oracle import mxfp4_ref as mx
from oracle import nvfp4_ref as o
from tests.experts_util import out_bytes, product_bound
from tests.gpu_util import dev, host, say

pytestmark = pytest.mark.gpu
RULES = [nv.MX_FLOOR, nv.MX_CEIL]


def values(seed, R, K):
    """fp32 values over many magnitudes, whole blocks of zeros and of special values among them."""
    rng = np.random.default_rng(seed)
    v = (rng.standard_normal((R, K)) * np.exp2(rng.integers(-20, 20, (R, K // 32))).repeat(32, 1)).astype(np.float32)
    v[rng.random((R, K)) < 0.05] = -0.0
    v[0, :32] = 0.0
    return v


def special(bf16: bool):
    inf, nan, big, tiny = np.inf, np.nan, 3.0e38, 2.0 ** -149
    rows = np.zeros((12, 64), np.float32)
    rows[0, 3], rows[1, 40], rows[2, 0] = nan, -nan, inf
    rows[3, 31], rows[3, 32] = -inf, nan
    rows[4, :] = big
    rows[5, :] = -big * np.linspace(0, 1, 64)
    rows[6, :] = tiny * np.arange(64)
    rows[7, :] = 2.0 ** -126 * np.linspace(-2, 2, 64)
    rows[8, :] = np.linspace(-6, 6, 64)
    rows[9, :] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25] * 8
    rows[10, :] = np.nextafter(np.float32(6), np.float32(7))
    rows[11, :32], rows[11, 32:] = -0.0, 1.9375
    return torch.from_numpy(rows).to(torch.bfloat16).float().numpy() if bf16 else rows


@pytest.mark.parametrize("rule", RULES)
@pytest.mark.parametrize("R,K", [(1, 32), (3, 64), (7, 96), (1, 6144), (33, 2080), (300, 768), (1025, 1024)])
def test_fp32_bit_for_bit(R, K, rule):
    say("mx quantize", R, K, rule)
    v = values(R + K, R, K)
    q, sf = out_bytes(R, K, 2), out_bytes(R, K, 32)
    nv.nvfp4_mx_quantize(dev(v), R, K, rule, q, sf)
    want = x.quantize(v, rule)
    np.testing.assert_array_equal(host(sf), want[1])
    np.testing.assert_array_equal(host(q), want[0])


@pytest.mark.parametrize("rule", RULES)
def test_special_values(rule):
    for bf16 in (False, True):
        v = special(bf16)
        R, K = v.shape
        q, sf = out_bytes(R, K, 2), out_bytes(R, K, 32)
        if bf16:
            nv.nvfp4_mx_quantize_rows_bf16(dev(v).bfloat16(), None, rule, q, sf, R, R, K)
        else:
            nv.nvfp4_mx_quantize(dev(v), R, K, rule, q, sf)
        want = x.quantize(v, rule)
        np.testing.assert_array_equal(host(sf), want[1])
        np.testing.assert_array_equal(host(q), want[0])


@pytest.mark.parametrize("rows,T,K", [(1, 1, 32), (5, 9, 32), (9, 4, 96), (64, 16, 256), (37, 5, 800), (500, 64, 6144),
                                      (3000, 7, 64), (2, 3, 8224)])
def test_gathered_rows_bit_for_bit(rows, T, K):
    say("mx quantize rows", rows, T, K)
    v = torch.from_numpy(values(rows, T, K)).to(torch.bfloat16)
    tok = np.random.default_rng(K).integers(-1, T + 1, rows).astype(np.int32)
    tok[0] = T - 1
    q, sf = out_bytes(rows, K, 2), out_bytes(rows, K, 32)
    for rule in RULES:
        nv.nvfp4_mx_quantize_rows_bf16(v.cuda(), dev(tok), rule, q, sf, rows, T, K)
        picked = np.where(((tok >= 0) & (tok < T))[:, None], v.float().numpy()[np.clip(tok, 0, T - 1)], 0.0)
        want = x.quantize(picked, rule)
        np.testing.assert_array_equal(host(sf), want[1])
        np.testing.assert_array_equal(host(q), want[0])
        n = min(rows, T)
        nv.nvfp4_mx_quantize_rows_bf16(v.cuda(), None, rule, q, sf, n, T, K)
        want = x.quantize(v.float().numpy()[:n], rule)
        np.testing.assert_array_equal(host(sf)[:n], want[1])
        np.testing.assert_array_equal(host(q)[:n], want[0])


@pytest.mark.parametrize("rule", RULES)
def test_quantised_product(rule):
    # activations and weights quantised and multiplied, against the same values in fp64
    M, N, K = 37, 65, 768
    rng = np.random.default_rng(8)
    a = torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).to(torch.bfloat16)
    b = (rng.standard_normal((N, K)) * 0.02).astype(np.float32)
    qa, sa, qb, sb = out_bytes(M, K, 2), out_bytes(M, K, 32), out_bytes(N, K, 2), out_bytes(N, K, 32)
    nv.nvfp4_mx_quantize_rows_bf16(a.cuda(), None, rule, qa, sa, M, M, K)
    nv.nvfp4_mx_quantize(dev(b), N, K, rule, qb, sb)
    d = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_mx_gemm(qa, sa, qb, sb, None, d, M, N, K, nv.mx_gemm_workspace(M, N, K))
    xa, xb = mx.dequant(*x.quantize(a.float().numpy(), rule)), mx.dequant(*x.quantize(b, rule))
    s = xa @ xb.T
    assert (np.abs(d.double().cpu().numpy() - s) <= product_bound(s, np.abs(xa) @ np.abs(xb).T, K)).all()
    # and near the unquantised product: each operand's error is below 1/4 of its block's peak
    full = a.double().numpy() @ b.astype(np.float64).T
    assert np.linalg.norm(s - full) / np.linalg.norm(full) < 0.25


def test_refused_tensors():
    v, q, sf = torch.zeros(4, 64, device="cuda"), out_bytes(4, 64, 2), out_bytes(4, 64, 32)
    nv.nvfp4_mx_quantize(v, 4, 64, 0, q, sf)
    tok = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in ((v.bfloat16(), 4, 64, 0, q, sf), (v, 5, 64, 0, q, sf), (v, 4, 64, 0, q[:3], sf), (v, 4, 64, 0, q, sf[:, :1]),
                (v, 4, 64, 2, q, sf), (v.cpu(), 4, 64, 0, q, sf), (v[:, :48], 4, 48, 0, q, sf)):
        with pytest.raises(nv.Nvfp4Error):
            nv.nvfp4_mx_quantize(*bad)
    h = v.bfloat16()
    nv.nvfp4_mx_quantize_rows_bf16(h, tok, 0, q, sf, 4, 4, 64)
    for bad in ((v, tok, 0, q, sf, 4, 4, 64), (h, tok.long(), 0, q, sf, 4, 4, 64), (h, tok[:3], 0, q, sf, 4, 4, 64),
                (h, None, 0, q, sf, 5, 4, 64), (h[:3], tok, 0, q, sf, 4, 4, 64), (h, tok, 0, q[:3], sf, 4, 4, 64)):
        with pytest.raises(nv.Nvfp4Error):
            nv.nvfp4_mx_quantize_rows_bf16(*bad)
