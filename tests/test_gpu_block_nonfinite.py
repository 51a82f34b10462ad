"""NaN and infinities through the NVFP4 outputs of the block operators: a block
of 16 that holds a NaN has scale byte 0x7F (NaN) and codes 0 on every plan, so
that what reads it is NaN too; infinities saturate; every other block is what
it is without them."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_07_amd as nv
from oracle import block_ref as br
from oracle import nvfp4_ref as o
from tests.block_util import bf16, dev_bf16, operand, values
from tests.gpu_util import dev, host, say, scalar

pytestmark = pytest.mark.gpu

NAN_SCALE = 0x7F
ALPHAS = np.array([0.02, 0.03], np.float32)


def _new(M, n):
    return (torch.full((M, n // 2), 0xEE, dtype=torch.uint8, device="cuda"),
            torch.full((M, n // 16), 0xEE, dtype=torch.uint8, device="cuda"))


def _nan_blocks(q, sf, nan):
    """Blocks where `nan` [rows][n] holds one: scale byte 0x7F, codes 0; no other scale byte is 0x7F."""
    rows, n = nan.shape
    bad = nan.reshape(rows, n // 16, 16).any(2)
    np.testing.assert_array_equal(sf == NAN_SCALE, bad)
    assert (q.reshape(rows, n // 16, 8)[bad] == 0).all()
    return bad


# register tiles of every width, and each LDS tile
@pytest.mark.parametrize("kind", [-1, 9, 10, 12, 14, 15, 32])
@pytest.mark.parametrize("M,I,K", [(5, 144, 512), (300, 272, 512)])
def test_gated_quantize(kind, M, I, K, force_plan):
    if kind >= 0:
        force_plan(nv.FAMILY_GEMM, kind, 0)
    say("nan gated", M, I, K, kind, nv.nvfp4_gemm_gated_plan(M, I, K))
    rng = np.random.default_rng(M + I)
    (a, asf, xa), (b, bsf, xb) = operand(1, M, K), operand(3, 2 * I, K)
    asf[1] = NAN_SCALE  # row 1 of A: NaN
    bias = bf16(rng.standard_normal(2 * I))
    bias[3] = np.nan                # one gate column of block 0
    bias[I + 16:I + 32] = np.nan    # all up columns of block 1
    bias[32 + 5] = np.inf           # an infinite gate: act(inf) * u is +-inf, saturated
    q, sf = _new(M, I)
    gs = np.float32(4.0)
    nv.nvfp4_gemm_gated_quantize(dev(a), dev(asf), dev(b), dev(bsf), dev(ALPHAS), dev_bf16(bias), nv.ACT_SILU, scalar(gs),
                                 q, sf, M, I, K, nv.gemm_gated_workspace(M, I, K))
    q, sf = host(q), host(sf)
    nan = np.zeros((M, I), bool)
    nan[1] = nan[:, 3] = nan[:, 16:32] = True
    _nan_blocks(q, sf, nan)
    rows = np.delete(np.arange(M), 1)
    # block 2 (infinity): the largest scale, and the infinite column's code is 6 with the sign of u
    finite = np.where(np.isfinite(bias), bias, np.float32(0.0))
    y, err = br.gated(xa, xb[:I], xb[I:], ALPHAS, finite, nv.ACT_SILU)
    assert (sf[rows, 2] == 0x7E).all()
    code = q[rows, (32 + 5) // 2] >> 4
    up = ALPHAS[1] * (xa @ xb[I + 37]) + bias[I + 37]
    np.testing.assert_array_equal(code, np.where(up[rows] < 0, 15, 7))
    # the others
    h, e = y[rows, 48:], err[rows, 48:]
    br.check_quantized(q[rows, 24:], sf[rows, 3:], h, e, gs, f"kind {kind}")


# row lengths of one wave, of several, with several chunks a thread, and past the registers
@pytest.mark.parametrize("T,H", [(5, 16), (5, 512), (6, 1040), (4, 6144), (600, 6144), (4, 20016)])
@pytest.mark.parametrize("kind", [nv.NORM_RMS, nv.NORM_LAYER])
def test_norm(T, H, kind):
    say("nan norm", T, H, kind)
    rng = np.random.default_rng(T + H)
    x, w = bf16(rng.standard_normal((T, H)) * 2), bf16(rng.standard_normal(H) * 0.2 + 1)
    x[1, H - 3] = np.nan
    x[2, 5] = np.inf
    gs = np.float32(100.0)
    q, sf = _new(T, H)
    y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    run = lambda q, sf, w: nv.nvfp4_residual_norm(dev_bf16(x), None, None, None, 0, None, 1.0, w, None, 1e-6, kind, None, y,
                                                  scalar(gs), q, sf, T, H)
    run(q, sf, dev_bf16(w))
    with np.errstate(invalid="ignore"):
        _, y32 = br.residual_norm(x, None, None, None, 0, None, 1.0, w, None, 1e-6, kind)
    nan = np.isnan(y32)
    assert nan[1].all() and nan[2].any() and not nan[[0, 3]].any()
    np.testing.assert_array_equal(np.isnan(values(y)), nan)
    bad = _nan_blocks(host(q), host(sf), nan)
    rq, rsf = o.quantize(np.where(np.repeat(bad, 16, 1), np.float32(0), y32), gs)
    np.testing.assert_array_equal(host(sf)[~bad], rsf[~bad])
    same = lambda c: c.reshape(T, H // 16, 8)[~bad]
    np.testing.assert_array_equal(same(host(q)), same(rq))
    # one NaN weight: the block of its column in every finite row
    w[H // 2] = np.nan
    run(q, sf, dev_bf16(w))
    assert (host(sf)[0] == NAN_SCALE).sum() == 1 and host(sf)[0, H // 2 // 16] == NAN_SCALE


@pytest.mark.parametrize("M", [1, 16, 100, 300, 1500])
def test_ffn_keeps_nan_in_its_row(M):
    H, I = 512, 1024
    say("nan ffn", M, nv.nvfp4_gemm_gated_plan(M, I, H), nv.nvfp4_gemm_epilogue_plan(M, H, I))
    (a, asf, _), (gu, gusf, _), (dn, dnsf, _) = operand(1, M, H), operand(3, 2 * I, H), operand(5, H, I)
    res = dev_bf16(bf16(np.random.default_rng(M).standard_normal((M, H))))
    ws = nv.ffn_workspace(M, H, I)
    w = dev(gu), dev(gusf), dev(ALPHAS), None, nv.ACT_SILU, scalar(2.0), dev(dn), dev(dnsf), scalar(1e-4), None

    def run(scales):
        d = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")
        return values(nv.nvfp4_ffn(dev(a), dev(scales), *w, res, 1.0, d, M, H, I, ws))
    want = run(asf)
    assert np.isfinite(want).all()
    bad = asf.copy()
    bad[M // 2, 7] = NAN_SCALE  # 16 elements of one token
    got = run(bad)
    assert np.isnan(got[M // 2]).all()
    others = np.delete(np.arange(M), M // 2)
    np.testing.assert_array_equal(got[others], want[others])
