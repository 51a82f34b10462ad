"""The 128- and 256-row LDS tiles of the block operators where the library
itself chooses them: every element against the formula at sizes with partial
tiles on both edges and a partial last band of tile rows (bands are 8 tiles
high), twice and captured with the same bits."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_07_amd as nv
from oracle import block_ref as br
from tests.block_util import bf16, close, dev_bf16, operand, values
from tests.gpu_util import dev, host, say, scalar

pytestmark = pytest.mark.gpu

ALPHA = np.float32(0.01)


def _three_times(call, outs):
    """The outputs of one call, of a second and of a replayed capture: equal bits."""
    call()
    first = [t.clone() for t in outs]
    call()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(2):
        for t in outs:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, outs))


@pytest.mark.parametrize("M,N,K,plan", [(2300, 6147, 512, "tile256x256w8k256_mfma32"), (1800, 4099, 512, "tile128x128k256_mfma32"),
                                        (2049, 5001, 512, "tile256x192w8k256_mfma32"), (5000, 2003, 256, "tile256x192w8k256_mfma32")])
@pytest.mark.parametrize("act,bias,residual", [(nv.ACT_GELU_TANH, True, True), (nv.ACT_NONE, False, False)])
def test_epilogue(M, N, K, plan, act, bias, residual):
    assert nv.nvfp4_gemm_epilogue_plan(M, N, K) == plan
    assert nv.nvfp4_gemm_epilogue_workspace_size(M, N, K) == 0
    say("epilogue", M, N, K, plan, act, bias, residual)
    rng = np.random.default_rng(M)
    (a, asf, xa), (b, bsf, xb) = operand(M, M, K), operand(N, N, K)
    bv = bf16(rng.standard_normal(N)) if bias else None
    rv = bf16(rng.standard_normal((M, N)) * 3) if residual else None
    ops = dev(a), dev(asf), dev(b), dev(bsf), scalar(ALPHA), None if bv is None else dev_bf16(bv), act
    res = None if rv is None else dev_bf16(rv)
    # rows 5 columns apart from each other, from an odd base: padding on all sides
    flat = torch.full((M * (N + 5) + 8,), -5.0, dtype=torch.bfloat16, device="cuda")
    d = flat[3:3 + M * (N + 5)].view(M, N + 5)[:, :N]
    _three_times(lambda: nv.nvfp4_gemm_epilogue(*ops, res, 0.75, d, M, N, K), [d])
    y, err = br.epilogue(xa, xb, ALPHA, bv, act, rv, 0.75)
    close(values(d), y, br.bf16_bound(y, err), plan)
    d.fill_(-5.0)
    assert bool((flat == -5.0).all()), "padding was written"
    if residual:
        nv.nvfp4_gemm_epilogue(*ops, res, 0.75, res, M, N, K)  # in place
        close(values(res), y, br.bf16_bound(y, err), plan + " in place")


@pytest.mark.parametrize("M,I,K,plan", [(1025, 6147, 512, "gated256x128w8"), (2300, 3008, 512, "gated256x128w8"),
                                        (2300, 9001, 256, "gated128x64"), (2300, 9008, 512, "gated128x64")])
def test_gated(M, I, K, plan):
    assert nv.nvfp4_gemm_gated_plan(M, I, K) == plan
    assert nv.nvfp4_gemm_gated_workspace_size(M, I, K) == 0
    say("gated", M, I, K, plan)
    rng = np.random.default_rng(M + I)
    (a, asf, xa), (b, bsf, xb) = operand(M, M, K), operand(I, 2 * I, K)
    bv, al = bf16(rng.standard_normal(2 * I)), np.array([ALPHA, 1.5 * ALPHA], np.float32)
    ops = dev(a), dev(asf), dev(b), dev(bsf), dev(al), dev_bf16(bv), nv.ACT_SILU
    h = torch.empty(M, I, dtype=torch.bfloat16, device="cuda")
    _three_times(lambda: nv.nvfp4_gemm_gated(*ops, h, M, I, K), [h])
    y, err = br.gated(xa, xb[:I], xb[I:], al, bv, nv.ACT_SILU)
    close(values(h), y, br.bf16_bound(y, err), plan)
    if I % 16:
        return
    gs = np.float32(2688.0 / np.abs(y).max())
    q = torch.empty(M, I // 2, dtype=torch.uint8, device="cuda")
    sf = torch.empty(M, I // 16, dtype=torch.uint8, device="cuda")
    gst = scalar(gs)
    _three_times(lambda: nv.nvfp4_gemm_gated_quantize(*ops, gst, q, sf, M, I, K), [q, sf])
    br.check_quantized(host(q), host(sf), y, err, gs, plan)


# prompt chunks through the feed-forward half: the 256-row tiles of both projections, with a full and a partial last band
@pytest.mark.parametrize("M,H,I", [(2048, 6144, 4096), (2300, 6144, 3584)])
def test_norm_and_feed_forward_repeat(M, H, I):
    plans = nv.nvfp4_gemm_gated_plan(M, I, H), nv.nvfp4_gemm_epilogue_plan(M, H, I)
    assert plans[0] == "gated256x128w8" and plans[1].startswith("tile256x")
    say("feed-forward", M, H, I, *plans)
    u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, H, device="cuda", generator=g).bfloat16()
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    (gu, gusf, _), (dn, dnsf, _) = operand(1, 2 * I, H), operand(2, H, I)
    weights = dev(gu), dev(gusf), dev(np.array([1e-4, 1e-4], np.float32)), None, nv.ACT_SILU, scalar(100.0), dev(dn), dev(dnsf), scalar(1e-5), None
    q, sf, r, d, gs = u8(M, H // 2), u8(M, H // 16), torch.empty_like(x), torch.empty_like(x), scalar(400.0)
    ws = nv.ffn_workspace(M, H, I)

    def half():
        nv.nvfp4_residual_norm(x, None, None, None, 0, x, 1.0, w, None, 1e-6, nv.NORM_RMS, r, None, gs, q, sf, M, H)
        nv.nvfp4_ffn(q, sf, *weights, r, 1.0, d, M, H, I, ws)
    _three_times(half, [r, q, sf, d])
    assert bool(torch.isfinite(d).all()) and not torch.equal(r, d)
