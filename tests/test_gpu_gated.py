"""nvfp4_gemm_gated, nvfp4_gemm_gated_quantize and nvfp4_ffn on the GPU through
the C ABI, against the formulas in fp64 at the bound of the kernel's roundings
(oracle.block_ref): bf16 and NVFP4 outputs, every plan, odd widths, strides,
biases, separate factors of gate and up, the feed-forward against its two
steps bit for bit and against the oracle's chain."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_07_amd as nv
from oracle import block_ref as br
from oracle import nvfp4_ref as o
from tests.block_util import bf16, close, dev_bf16, operand, values
from tests.gpu_util import bits, dev, host, say, scalar

pytestmark = pytest.mark.gpu

ALPHAS = np.array([0.02, 0.03], np.float32)


def _case(M, I, K, seed, bias):
    rng = np.random.default_rng(seed)
    a, asf, xa = operand(seed + 1, M, K)
    b, bsf, xb = operand(seed + 3, 2 * I, K)
    bv = bf16(rng.standard_normal(2 * I)) if bias else None
    return (dev(a), dev(asf), dev(b), dev(bsf)), xa, xb, bv


def _alphas(K):
    return (ALPHAS / np.sqrt(K / 256)).astype(np.float32)


def _check(M, I, K, seed, act=nv.ACT_SILU, bias=False, label=""):
    ops, xa, xb, bv = _case(M, I, K, seed, bias)
    al = _alphas(K)
    ws = nv.gemm_gated_workspace(M, I, K)
    h = torch.full((M, I), 777.0, dtype=torch.bfloat16, device="cuda")
    say("gated", M, I, K, nv.nvfp4_gemm_gated_plan(M, I, K), "act", act, bias, label)
    out = nv.nvfp4_gemm_gated(*ops, dev(al), None if bv is None else dev_bf16(bv), act, h, M, I, K, ws)
    assert out is h
    y, err = br.gated(xa, xb[:I], xb[I:], al, bv, act)
    close(values(h), y, br.bf16_bound(y, err), f"{M}x{I}x{K}")
    if I % 16 == 0:
        gs = np.float32(2688.0 / np.abs(y).max())
        q = torch.full((M, I // 2), 0xEE, dtype=torch.uint8, device="cuda")
        sf = torch.full((M, I // 16), 0xEE, dtype=torch.uint8, device="cuda")
        nv.nvfp4_gemm_gated_quantize(*ops, dev(al), None if bv is None else dev_bf16(bv), act, scalar(gs), q, sf, M, I,
                                     K, ws)
        br.check_quantized(host(q), host(sf), y, err, gs, f"{M}x{I}x{K}")


@pytest.mark.parametrize("M,I,K", [(1, 2048, 512), (1, 16, 256), (1, 4112, 256), (16, 9008, 512), (16, 2048, 6144), (5, 33, 256), (31, 4096, 512),
                                   (64, 2048, 1024), (128, 4096, 512), (100, 784, 1280), (333, 1001, 1536),
                                   (513, 1040, 512), (1, 1, 256), (17, 3, 512), (70, 9, 256), (9, 2001, 2304), (3, 24, 1 << 20),
                                   (70, 40, 1 << 20)])
@pytest.mark.parametrize("bias", [False, True])
def test_shapes(M, I, K, bias):
    _check(M, I, K, 11 * M + I, bias=bias)


@pytest.mark.parametrize("act", [nv.ACT_NONE, nv.ACT_RELU, nv.ACT_GELU, nv.ACT_GELU_TANH, nv.ACT_SILU])
def test_activations(act):
    _check(37, 144, 512, 100 + act, act=act, bias=True)


@pytest.mark.parametrize("kind,splits", [(9, 0), (9, 3), (10, 0), (10, 2), (12, 0), (12, 3), (14, 0), (15, 0), (15, 4),
                                         (16, 0), (32, 0), (32, 2), (33, 0), (33, 3)])
@pytest.mark.parametrize("M,I,K", [(70, 272, 1536), (257, 99, 768)])
def test_every_plan_forced(kind, splits, M, I, K, force_plan):
    force_plan(nv.FAMILY_GEMM, kind, splits)
    _check(M, I, K, 17 * kind + splits + M, bias=True, label=f"kind {kind}/{splits}")


@pytest.mark.parametrize("M,I,K", [(4096, 2064, 256), (2048, 4096, 512), (1000, 4100, 512), (130, 16400, 256)])
def test_large_tiles(M, I, K):
    _check(M, I, K, M + I, bias=True)


def test_strides_padding_and_offsets():
    M, I, K = 45, 41, 512
    ops, xa, xb, bv = _case(M, I, K, 900, True)
    flat = torch.full((M * 50 + 8,), -5.0, dtype=torch.bfloat16, device="cuda")
    h = flat[3:3 + M * 50].view(M, 50)[:, :I]
    nv.nvfp4_gemm_gated(*ops, dev(_alphas(K)), dev_bf16(bv), nv.ACT_SILU, h, M, I, K, nv.gemm_gated_workspace(M, I, K))
    y, err = br.gated(xa, xb[:I], xb[I:], _alphas(K), bv, nv.ACT_SILU)
    close(values(h), y, br.bf16_bound(y, err), "strided")
    whole = host(flat.float())
    mask = np.ones(whole.size, dtype=bool)
    mask[(3 + np.arange(M)[:, None] * 50 + np.arange(I)[None, :]).reshape(-1)] = False
    assert (whole[mask] == -5.0).all(), "padding of h was written"


def test_no_alpha_and_all_zero_blocks():
    # zero scale bytes make whole blocks zero: scale 0, codes 0 (or -0)
    M, I, K = 20, 64, 256
    ops, xa, xb, _ = _case(M, I, K, 61, False)
    y, err = br.gated(xa, xb[:I], xb[I:], (1.0, 1.0), None, nv.ACT_NONE)
    h = torch.empty((M, I), dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_gemm_gated(*ops, None, None, nv.ACT_NONE, h, M, I, K, nv.gemm_gated_workspace(M, I, K))
    close(values(h), y, br.bf16_bound(y, err), "no alpha")
    ops[1].zero_()
    q = torch.full((M, I // 2), 0xEE, dtype=torch.uint8, device="cuda")
    sf = torch.full((M, I // 16), 0xEE, dtype=torch.uint8, device="cuda")
    nv.nvfp4_gemm_gated_quantize(*ops, None, None, nv.ACT_SILU, None, q, sf, M, I, K, nv.gemm_gated_workspace(M, I, K))
    assert (host(sf) == 0).all() and ((host(q) & 0x77) == 0).all()


def _ffn_case(M, H, I, seed, biases):
    rng = np.random.default_rng(seed)
    a, asf, xa = operand(seed + 1, M, H)
    gu, gusf, xgu = operand(seed + 3, 2 * I, H)
    dn, dnsf, xdn = operand(seed + 5, H, I)
    bgu = bf16(rng.standard_normal(2 * I)) if biases else None
    bd = bf16(rng.standard_normal(H)) if biases else None
    res = bf16(rng.standard_normal((M, H)) * 2)
    return dict(a=a, asf=asf, xa=xa, gu=gu, gusf=gusf, xgu=xgu, dn=dn, dnsf=dnsf, xdn=xdn, bgu=bgu, bd=bd, res=res)


@pytest.mark.parametrize("M,H,I", [(1, 512, 256), (7, 768, 2048), (64, 6144, 2048), (300, 512, 1024), (1500, 1024, 2048)])
@pytest.mark.parametrize("biases", [False, True])
def test_ffn_equals_its_steps_and_the_oracle(M, H, I, biases):
    c = _ffn_case(M, H, I, 31 * M + I, biases)
    al = _alphas(H)
    h64, _ = br.gated(c["xa"], c["xgu"][:I], c["xgu"][I:], al, c["bgu"], nv.ACT_SILU)
    gs = np.float32(2688.0 / np.abs(h64).max())
    ald = np.float32(1.0 / (gs * 40.0 * np.sqrt(I / 256)))
    opt = lambda v: None if v is None else dev_bf16(v)
    ops = [dev(c[k]) for k in ("a", "asf", "gu", "gusf")]
    bgu, bd, res = opt(c["bgu"]), opt(c["bd"]), dev_bf16(c["res"])
    dn, dnsf = dev(c["dn"]), dev(c["dnsf"])
    ws = nv.ffn_workspace(M, H, I)
    d = torch.empty((M, H), dtype=torch.bfloat16, device="cuda")
    say("ffn", M, H, I, nv.nvfp4_gemm_gated_plan(M, I, H), nv.nvfp4_gemm_epilogue_plan(M, H, I))
    out = nv.nvfp4_ffn(*ops, dev(al), bgu, nv.ACT_SILU, scalar(gs), dn, dnsf, scalar(ald), bd, res, 0.5, d, M, H, I, ws)
    assert out is d
    q = torch.empty((M, I // 2), dtype=torch.uint8, device="cuda")
    sf = torch.empty((M, I // 16), dtype=torch.uint8, device="cuda")
    step = torch.empty_like(d)
    nv.nvfp4_gemm_gated_quantize(*ops, dev(al), bgu, nv.ACT_SILU, scalar(gs), q, sf, M, I, H, nv.gemm_gated_workspace(M, I, H))
    nv.nvfp4_gemm_epilogue(q, sf, dn, dnsf, scalar(ald), bd, nv.ACT_NONE, res, 0.5, step, M, H, I,
                           nv.gemm_epilogue_workspace(M, H, I))
    np.testing.assert_array_equal(bits(d.view(torch.int16)), bits(step.view(torch.int16)))
    hq, hsf = o.quantize(h64.astype(np.float32), gs)
    y, _ = br.epilogue(o.dequant(hq, hsf), c["xdn"], ald, c["bd"], 0, c["res"], 0.5)
    frob = np.linalg.norm(values(d) - y) / np.linalg.norm(y)
    assert frob <= 1e-2, frob


def test_ffn_in_place_replays_and_shared_workspace():
    sizes = [(64, 512, 1024), (16, 6144, 2048), (64, 512, 1024)]
    ws = nv.nvfp4_workspace_init(torch.empty(max(nv.nvfp4_ffn_workspace_size(*s) for s in sizes), dtype=torch.uint8,
                                             device="cuda"))
    for M, H, I in sizes:
        c = _ffn_case(M, H, I, M + H, False)
        args = [dev(c["a"]), dev(c["asf"]), dev(c["gu"]), dev(c["gusf"]), dev(_alphas(H)), None, nv.ACT_GELU_TANH,
                scalar(4.0), dev(c["dn"]), dev(c["dnsf"]), scalar(1e-4), None]
        res = dev_bf16(c["res"])
        want = torch.empty_like(res)
        nv.nvfp4_ffn(*args, res, 1.0, want, M, H, I, ws)
        d = res.clone()
        nv.nvfp4_ffn(*args, d, 1.0, d, M, H, I, ws)
        assert torch.equal(d, want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            nv.nvfp4_ffn(*args, res, 1.0, d, M, H, I, ws)
        for i in range(3):
            d.fill_(float(i))
            nv.nvfp4_ffn(*args, res, 1.0, want, M, H, I, ws)
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(d, want), f"replay {i}"
    assert (host(ws[:4096]) == 0).all()
