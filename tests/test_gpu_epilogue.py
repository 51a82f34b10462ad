"""nvfp4_gemm_epilogue on the GPU through the C ABI, against the formula in
fp64 at the bound of the kernel's roundings (oracle.block_ref): every plan
family, activation, bias and residual combination, odd sizes, row strides,
in-place residuals, untouched padding, non-finite values, graph replays."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_07_amd as nv
from oracle import block_ref as br
from tests.block_util import bf16, close, dev_bf16, operand, values
from tests.gpu_util import bits, dev, gpu_gemm, host, say, scalar

pytestmark = pytest.mark.gpu

# alpha that brings sums of random codes to a few units
ALPHA = 0.02


def _case(M, N, K, seed, bias, residual):
    rng = np.random.default_rng(seed)
    a, asf, xa = operand(seed + 1, M, K)
    b, bsf, xb = operand(seed + 3, N, K)
    bv = bf16(rng.standard_normal(N)) if bias else None
    rv = bf16(rng.standard_normal((M, N)) * 3) if residual else None
    return (dev(a), dev(asf), dev(b), dev(bsf)), xa, xb, bv, rv


def _check(M, N, K, seed, act=nv.ACT_NONE, bias=False, residual=False, beta=1.0, label=""):
    ops, xa, xb, bv, rv = _case(M, N, K, seed, bias, residual)
    alpha = np.float32(ALPHA / np.sqrt(K / 256))
    ws = nv.gemm_epilogue_workspace(M, N, K)
    d = torch.full((M, N), 777.0, dtype=torch.bfloat16, device="cuda")
    say("epilogue", M, N, K, nv.nvfp4_gemm_epilogue_plan(M, N, K), "act", act, bias, residual, label)
    out = nv.nvfp4_gemm_epilogue(*ops, scalar(alpha), None if bv is None else dev_bf16(bv), act,
                                 None if rv is None else dev_bf16(rv), beta, d, M, N, K, ws)
    assert out is d
    y, err = br.epilogue(xa, xb, alpha, bv, act, rv, beta)
    close(values(d), y, br.bf16_bound(y, err), f"{M}x{N}x{K} act {act}")


# one shape per plan family, each odd in M or N where the family allows
SHAPES = [(1, 768, 512), (1, 6144, 2048), (16, 9000, 512), (16, 768, 6144), (5, 33, 256), (31, 4096, 512), (64, 2048, 1024), (128, 4096, 512),
          (61, 777, 1280), (200, 300, 768), (513, 1025, 512), (1, 1, 256), (17, 2, 768), (65, 7, 256), (300, 1, 512)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", [nv.ACT_NONE, nv.ACT_GELU])
def test_shapes(M, N, K, act):
    _check(M, N, K, 11 * M + N, act=act, bias=True, residual=True, beta=0.75)


@pytest.mark.parametrize("act", [nv.ACT_NONE, nv.ACT_RELU, nv.ACT_GELU, nv.ACT_GELU_TANH, nv.ACT_SILU])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True), (True, True)])
def test_activations_bias_and_residual(act, bias, residual):
    _check(37, 136, 512, 100 + act, act=act, bias=bias, residual=residual, beta=-1.5)


@pytest.mark.parametrize("kind,splits", [(9, 0), (9, 3), (10, 0), (10, 2), (11, 0), (11, 2), (12, 0), (12, 3), (14, 0),
                                         (15, 0), (15, 4), (16, 0), (3, 2), (32, 0), (32, 3), (33, 0), (34, 0), (34, 1), (34, 3)])
@pytest.mark.parametrize("M,N,K", [(70, 270, 1536), (257, 195, 768)])
def test_every_plan_forced(kind, splits, M, N, K, force_plan):
    force_plan(nv.FAMILY_GEMM, kind, splits)
    _check(M, N, K, 17 * kind + splits + M, act=nv.ACT_SILU, bias=True, residual=True, label=f"kind {kind}/{splits}")


@pytest.mark.parametrize("M,N,K", [(8192, 6144, 256), (4096, 4100, 512), (2048, 6144, 256)])
def test_large_tiles(M, N, K):
    _check(M, N, K, M + N, act=nv.ACT_GELU_TANH, bias=True, residual=True)


@pytest.mark.parametrize("kind,splits", [(9, 1), (9, 4), (14, 0), (15, 0), (16, 0)])
@pytest.mark.parametrize("M,N,K", [(1, 768, 1024), (300, 1000, 1024), (1024, 256, 6144)])
def test_plain_call_equals_nvfp4_gemm_on_the_same_plan(kind, splits, M, N, K, force_plan):
    force_plan(nv.FAMILY_GEMM, kind, splits if kind == 9 else 1)
    ops, *_ = _case(M, N, K, 5 + M, False, False)
    d = torch.empty((M, N), dtype=torch.int16, device="cuda")
    nv.nvfp4_gemm_epilogue(*ops, scalar(0.5), None, nv.ACT_NONE, None, 0.0, d, M, N, K, nv.gemm_epilogue_workspace(M, N, K))
    np.testing.assert_array_equal(bits(d), bits(gpu_gemm(*ops, scalar(0.5), M, N, K)))


@pytest.mark.parametrize("M,N,ldr,ldd,off", [(19, 40, 48, 56, 0), (33, 41, 47, 43, 0), (70, 64, 80, 72, 1), (300, 136, 136, 144, 3)])
def test_row_strides_offsets_and_padding(M, N, ldr, ldd, off):
    # off shifts the bases by single elements: the 16-byte path must not be taken
    K, alpha = 512, np.float32(ALPHA)
    ops, xa, xb, bv, rv = _case(M, N, K, 900 + M, True, True)
    flat_r = torch.full((M * ldr + 8,), float("nan"), dtype=torch.bfloat16, device="cuda")
    flat_d = torch.full((M * ldd + 8,), -5.0, dtype=torch.bfloat16, device="cuda")
    flat_b = torch.zeros(N + 8, dtype=torch.bfloat16, device="cuda")
    r = flat_r[off:off + M * ldr].view(M, ldr)[:, :N]
    d = flat_d[off:off + M * ldd].view(M, ldd)[:, :N]
    bias = flat_b[off:off + N]
    r.copy_(dev_bf16(rv))
    bias.copy_(dev_bf16(bv))
    say("strides", M, N, ldr, ldd, off)
    nv.nvfp4_gemm_epilogue(*ops, scalar(alpha), bias, nv.ACT_RELU, r, 2.0, d, M, N, K, nv.gemm_epilogue_workspace(M, N, K))
    y, err = br.epilogue(xa, xb, alpha, bv, nv.ACT_RELU, rv, 2.0)
    close(values(d), y, br.bf16_bound(y, err), "strided")
    whole = host(flat_d.float())
    mask = np.ones(whole.size, dtype=bool)
    idx = off + np.arange(M)[:, None] * ldd + np.arange(N)[None, :]
    mask[idx.reshape(-1)] = False
    assert (whole[mask] == -5.0).all(), "padding of d was written"


@pytest.mark.parametrize("M", [5, 300])
def test_rows_past_32_bit_offsets(M):
    # the last row of d and residual starts past 2^33 bytes (register and LDS tiles)
    N, K, alpha = 40, 512, np.float32(ALPHA)
    ld = -(-(1 << 32) // (M - 1)) + 8
    ops, xa, xb, bv, rv = _case(M, N, K, 950, True, True)
    big = torch.empty((M - 1) * ld + 2 * N, dtype=torch.bfloat16, device="cuda")
    r, d = big.as_strided((M, N), (ld, 1), 0), big.as_strided((M, N), (ld, 1), N)
    r.copy_(dev_bf16(rv))
    nv.nvfp4_gemm_epilogue(*ops, scalar(alpha), dev_bf16(bv), 0, r, 1.0, d, M, N, K, nv.gemm_epilogue_workspace(M, N, K))
    y, err = br.epilogue(xa, xb, alpha, bv, 0, rv, 1.0)
    close(values(d), y, br.bf16_bound(y, err), "far rows")


@pytest.mark.parametrize("M,N,K", [(3, 768, 512), (16, 768, 6144), (64, 768, 6144), (512, 768, 6144), (700, 1000, 512)])
def test_residual_in_place(M, N, K):
    ops, xa, xb, _, rv = _case(M, N, K, 40 + M, False, True)
    d = dev_bf16(rv)
    ws = nv.gemm_epilogue_workspace(M, N, K)
    sep = torch.empty_like(d)
    nv.nvfp4_gemm_epilogue(*ops, scalar(ALPHA), None, nv.ACT_NONE, d, 1.0, sep, M, N, K, ws)
    nv.nvfp4_gemm_epilogue(*ops, scalar(ALPHA), None, nv.ACT_NONE, d, 1.0, d, M, N, K, ws)
    assert torch.equal(sep, d)


def test_no_alpha_beta_zero_and_non_finite_residual():
    M, N, K = 20, 48, 256
    ops, xa, xb, _, rv = _case(M, N, K, 77, False, True)
    y, err = br.epilogue(xa, xb, 1.0, None, 0, rv, 0.0)
    d = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_gemm_epilogue(*ops, None, None, 0, dev_bf16(rv), 0.0, d, M, N, K)
    close(values(d), y, br.bf16_bound(y, err), "beta 0")
    rv[3, 5], rv[4, 6], rv[5, 7] = np.inf, -np.inf, np.nan
    nv.nvfp4_gemm_epilogue(*ops, None, None, 0, dev_bf16(rv), 1.0, d, M, N, K)
    got = values(d)
    assert got[3, 5] == np.inf and got[4, 6] == -np.inf and np.isnan(got[5, 7])
    assert np.isfinite(np.delete(got.reshape(-1), [3 * N + 5, 4 * N + 6, 5 * N + 7])).all()


@pytest.mark.parametrize("act", [1, 2, 3, 4])
def test_activations_at_large_arguments(act):
    # a bias of +-60000 drives the activation to its limits; NaN stays NaN
    M, N, K = 4, 32, 256
    ops, xa, xb, _, _ = _case(M, N, K, 55, False, False)
    bv = np.zeros(N, np.float32)
    bv[0], bv[1], bv[2], bv[3] = 60160.0, -60160.0, 1e30, -1e30
    bv[4] = np.nan
    d = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_gemm_epilogue(*ops, scalar(ALPHA), dev_bf16(bf16(bv)), act, None, 0.0, d, M, N, K)
    got = values(d)
    assert (np.abs(got[:, 0] / 60160.0 - 1) < 0.01).all() and (np.abs(got[:, 2] / 1e30 - 1) < 0.01).all()
    assert (got[:, 1] == 0).all() and (got[:, 3] == 0).all() and np.isnan(got[:, 4]).all()


def test_workspace_serves_any_shape_and_results_repeat():
    shapes = [(1024, 768, 6144), (16, 768, 6144), (512, 768, 2048), (64, 512, 8192), (1024, 768, 6144)]
    assert sum(nv.nvfp4_gemm_epilogue_workspace_size(*s) > 0 for s in shapes) == 4
    need = max(nv.nvfp4_gemm_epilogue_workspace_size(*s) for s in shapes)
    ws = nv.nvfp4_workspace_init(torch.empty(need, dtype=torch.uint8, device="cuda"))
    first = {}
    for M, N, K in shapes * 2:
        ops, _, _, bv, rv = _case(M, N, K, 7 * M + K, True, True)
        d = torch.empty((M, N), dtype=torch.int16, device="cuda")
        nv.nvfp4_gemm_epilogue(*ops, scalar(ALPHA), dev_bf16(bv), nv.ACT_SILU, dev_bf16(rv), 1.0, d, M, N, K, ws)
        got = bits(d)
        np.testing.assert_array_equal(first.setdefault((M, N, K), got), got)
    assert (host(ws[:4096]) == 0).all(), "counters are back at zero"


def test_graph_replays_and_another_stream():
    M, N, K = 16, 768, 6144
    ops, xa, xb, bv, rv = _case(M, N, K, 321, True, True)
    bias, res, alpha = dev_bf16(bv), dev_bf16(rv), scalar(ALPHA)
    ws = nv.gemm_epilogue_workspace(M, N, K)
    want = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    d = torch.empty_like(want)
    call = lambda out: nv.nvfp4_gemm_epilogue(*ops, alpha, bias, nv.ACT_GELU, res, 1.0, out, M, N, K, ws)
    call(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(d)
    torch.cuda.synchronize()
    assert torch.equal(d, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(d)
    for i in range(4):
        d.fill_(float(i))
        res.mul_(-1.0)
        call(want)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(d, want), f"replay {i}"


def test_refused_tensors_leave_the_output_alone():
    M, N, K = 4, 32, 256
    ops, *_ = _case(M, N, K, 5, False, False)
    d = torch.full((M, N), 3.0, dtype=torch.bfloat16, device="cuda")
    call = lambda *a, **k: nv.nvfp4_gemm_epilogue(*a, **k)
    base = [*ops, None, None, 0, None, 0.0, d, M, N, K]
    half = torch.zeros(M, N, dtype=torch.float16, device="cuda")
    wide = torch.zeros(M, 2 * N, dtype=torch.bfloat16, device="cuda")
    bad = [(0, ops[0].cpu()), (0, ops[0][:2]), (2, ops[2].t()), (4, half.double()), (5, half[0]), (7, half), (9, half),
           (7, wide), (9, wide[:, ::2]), (9, d[:3]), (9, d.t()), (9, d[:1].expand(M, N)), (9, np.zeros((M, N))),
           (7, torch.zeros(M, N, device="meta", dtype=torch.bfloat16)), (6, 17), (10, -4)]
    for i, v in bad:
        args = list(base)
        args[i] = v
        with pytest.raises(nv.Nvfp4Error):
            call(*args)
    # a tensor without storage raises, it does not end the process
    with pytest.raises((nv.Nvfp4Error, RuntimeError)):
        call(*[d.to_sparse() if i == 9 else v for i, v in enumerate(base)])
    for args in ([*base[:-1], "256"], [*base[:8], "x", *base[9:]]):
        with pytest.raises(TypeError):
            call(*args)
    torch.cuda.synchronize()
    assert (d == 3.0).all()


def test_two_calls_at_once_on_two_streams():
    M, N, K = 16, 768, 6144
    cases = [_case(M, N, K, s, True, True) for s in (71, 72)]
    streams = [torch.cuda.Stream() for _ in cases]
    args, want, got = [], [], []
    for ops, _, _, bv, rv in cases:
        args.append((*ops, scalar(ALPHA), dev_bf16(bv), nv.ACT_GELU, dev_bf16(rv), 1.0))
        want.append(nv.nvfp4_gemm_epilogue(*args[-1], torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), M, N, K,
                                           nv.gemm_epilogue_workspace(M, N, K)))
        got.append(torch.empty(M, N, dtype=torch.bfloat16, device="cuda"))
    spaces = [nv.gemm_epilogue_workspace(M, N, K) for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for a, s, d, ws in zip(args, streams, got, spaces):
            nv.nvfp4_gemm_epilogue(*a, d, M, N, K, ws, stream=s.cuda_stream)
    torch.cuda.synchronize()
    for d, w in zip(got, want):
        assert torch.equal(d, w)


@pytest.mark.parametrize("M,N,kind", [(3, 40, -1), (70, 72, 9), (70, 72, 34), (40, 40, 14)])
def test_long_k(M, N, kind, force_plan):
    # 2^20 terms a sum; operand rows of 512 KB
    if kind >= 0:
        force_plan(nv.FAMILY_GEMM, kind, 0)
    _check(M, N, 1 << 20, 5, act=nv.ACT_NONE, bias=True, residual=True)
