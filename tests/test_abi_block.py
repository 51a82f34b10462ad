"""Host-side refusals, sizes and no-ops of the block operators (CPU only:
every call is answered before any HIP call)."""
import pytest

import nvfp4_block_scaled_07_amd as nv

FAKE = 0x10000  # an aligned non-NULL address; never dereferenced
NULL, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5


def _call(fn, defaults, kw):
    args = {**defaults, **kw}
    assert set(args) == set(defaults)
    return getattr(nv.lib(), fn)(*args.values())


def _epi(**kw):
    return _call("nvfp4_gemm_epilogue", dict(a=FAKE, a_sf=FAKE, b=FAKE, b_sf=FAKE, alpha=None, bias=None, act=0,
                                             residual=None, ldr=0, beta=1.0, d=FAKE, ldd=0, M=16, N=16, K=256, ws=None,
                                             wsb=0, stream=None), kw)


def _gated(**kw):
    return _call("nvfp4_gemm_gated", dict(a=FAKE, a_sf=FAKE, b=FAKE, b_sf=FAKE, alpha=None, bias=None, act=0, h=FAKE,
                                          ldh=0, M=16, I=16, K=256, ws=None, wsb=0, stream=None), kw)


def _gatedq(**kw):
    return _call("nvfp4_gemm_gated_quantize", dict(a=FAKE, a_sf=FAKE, b=FAKE, b_sf=FAKE, alpha=None, bias=None, act=0,
                                                   gs=None, q=FAKE, sf=FAKE, M=16, I=16, K=256, ws=None, wsb=0,
                                                   stream=None), kw)


def _ffn(**kw):
    return _call("nvfp4_ffn", dict(a=FAKE, a_sf=FAKE, gu=FAKE, gu_sf=FAKE, al=None, bgu=None, act=4, gs=None, dn=FAKE,
                                   dn_sf=FAKE, ald=None, bd=None, residual=None, ldr=0, beta=1.0, d=FAKE, ldd=0, M=16,
                                   H=256, I=256, ws=FAKE, wsb=0, stream=None), kw)


def _norm(**kw):
    return _call("nvfp4_residual_norm", dict(x=FAKE, ldx=0, post_w=None, post_b=None, gate=None, group=0, res=None,
                                             ldres=0, beta=1.0, w=None, b=None, eps=1e-6, kind=0, r=None, ldr=0, y=FAKE,
                                             ldy=0, gs=None, q=None, sf=None, T=4, H=64, stream=None), kw)


@pytest.mark.parametrize("call,cols", [(_epi, "N"), (_gated, "I"), (_gatedq, "I")])
def test_gemm_refusals(call, cols):
    big = 1 << 41
    assert call(M=-1) == SHAPE and call(**{cols: -16}) == SHAPE
    assert call(K=40) == SHAPE and "block size 16" in nv.nvfp4_last_error()
    assert call(K=128) == UNSUPPORTED and call(K=0) == UNSUPPORTED and call(K=(1 << 22) + 256) == UNSUPPORTED
    assert call(act=5) == SHAPE and "act" in nv.nvfp4_last_error()
    assert call(act=-1) == SHAPE
    for name in ("a", "a_sf", "b", "b_sf"):
        assert call(**{name: None}) == NULL
        assert call(**{name: FAKE + 8}) == ALIGN
    assert call(alpha=FAKE + 2) == ALIGN and call(bias=FAKE + 1) == ALIGN
    assert call(M=big) == UNSUPPORTED and call(M=1 << 22, **{cols: 1 << 22}) == UNSUPPORTED
    assert call(M=0, a=None, b=None) == 0 and call(**{cols: 0}) == 0
    assert nv.nvfp4_last_error() == ""


def test_epilogue_refusals():
    assert _epi(d=None) == NULL and _epi(d=FAKE + 1) == ALIGN and _epi(residual=FAKE + 1) == ALIGN
    assert _epi(ldd=15) == SHAPE and "ldd" in nv.nvfp4_last_error()
    assert _epi(residual=FAKE, ldr=15) == SHAPE and "ldr" in nv.nvfp4_last_error()
    assert _epi(residual=FAKE, ldr=-1) == SHAPE
    need = nv.nvfp4_gemm_epilogue_workspace_size(1024, 768, 6144)
    assert need > 0
    shape = dict(M=1024, N=768, K=6144)
    assert _epi(**shape) == WORKSPACE and "workspace" in nv.nvfp4_last_error()
    assert _epi(**shape, ws=FAKE, wsb=need - 1) == WORKSPACE
    assert _epi(**shape, ws=FAKE + 16, wsb=need) == ALIGN


def test_gated_refusals():
    assert _gated(h=None) == NULL and _gated(h=FAKE + 1) == ALIGN and _gated(ldh=8) == SHAPE
    assert _gatedq(I=40) == SHAPE and _gatedq(q=None) == NULL and _gatedq(sf=None) == NULL
    assert _gatedq(q=FAKE + 4) == ALIGN and _gatedq(gs=FAKE + 2) == ALIGN
    need = nv.nvfp4_gemm_gated_workspace_size(16, 2048, 6144)
    assert need > 0
    assert _gatedq(I=2048, K=6144) == WORKSPACE
    assert _gatedq(I=2048, K=6144, ws=FAKE, wsb=need - 1) == WORKSPACE
    need = nv.nvfp4_gemm_gated_workspace_size(256, 2048, 6144)
    assert need > 0
    assert _gated(M=256, I=2048, K=6144) == WORKSPACE
    assert _gated(M=256, I=2048, K=6144, ws=FAKE, wsb=need - 1) == WORKSPACE


def test_ffn_refusals():
    need = nv.nvfp4_ffn_workspace_size(16, 256, 256)
    assert need >= 4096 + 16 * 128 + 16 * 16
    assert _ffn(wsb=need - 1) == WORKSPACE and _ffn(ws=None, wsb=need) == WORKSPACE
    assert _ffn(ws=FAKE + 128, wsb=need) == ALIGN
    assert _ffn(H=384) == UNSUPPORTED and _ffn(I=384) == UNSUPPORTED and _ffn(I=8) == SHAPE
    for name in ("a", "a_sf", "gu", "gu_sf", "dn", "dn_sf", "d"):
        assert _ffn(**{name: None}) == NULL, name
    assert _ffn(act=9) == SHAPE and _ffn(residual=FAKE, ldr=255) == SHAPE and _ffn(ldd=100) == SHAPE
    assert _ffn(gs=FAKE + 1) == ALIGN and _ffn(ald=FAKE + 1) == ALIGN and _ffn(bd=FAKE + 1) == ALIGN
    assert _ffn(M=0, a=None) == 0
    assert nv.nvfp4_ffn_workspace_size(16, 100, 256) == 0


def test_norm_refusals():
    assert _norm(T=-1) == SHAPE and _norm(H=0) == SHAPE and _norm(kind=2) == SHAPE and _norm(group=-1) == SHAPE
    assert _norm(eps=-1e-6) == SHAPE and _norm(eps=float("nan")) == SHAPE
    assert _norm(x=None) == NULL and _norm(y=None) == NULL and "no output" in nv.nvfp4_last_error()
    assert _norm(q=FAKE) == NULL and _norm(sf=FAKE) == NULL and _norm(post_b=FAKE) == NULL
    assert _norm(q=FAKE, sf=FAKE, H=72) == SHAPE and _norm(q=FAKE + 4, sf=FAKE) == ALIGN
    for name in ("ldx", "ldres", "ldr", "ldy"):
        assert _norm(**{name: 63}) == SHAPE
    for name in ("x", "post_w", "gate", "res", "w", "b", "r", "y"):
        assert _norm(**{name: FAKE + 1}) == ALIGN
    assert _norm(gs=FAKE + 2, q=FAKE, sf=FAKE) == ALIGN
    assert _norm(T=1 << 31) == UNSUPPORTED and _norm(H=(1 << 30) + 1) == UNSUPPORTED
    assert _norm(T=0, x=None, y=None) == 0


def test_queries():
    for M, N, K in [(8192, 6144, 6144), (2048, 6144, 16384), (4096, 8192, 2048)]:
        assert nv.nvfp4_gemm_epilogue_plan(M, N, K) == nv.nvfp4_gemm_plan(M, N, K)
        assert nv.nvfp4_gemm_epilogue_workspace_size(M, N, K) == nv.nvfp4_gemm_workspace_size(M, N, K) == 0
    for (M, N, K), plan in {(1, 768, 6144): "kreg16x16k8", (16, 6144, 2048): "kreg16x32k8", (64, 2048, 6144): "kreg32x16k8",
                            (256, 1024, 2048): "kreg32x32k8", (64, 768, 16384): "kreg32x32k8",
                            (128, 768, 16384): "tile64x64k4w8", (1024, 768, 6144): "tile64x64k4",
                            (4096, 4096, 6144): "tile256x256w8k256_mfma32", (1024, 8192, 2048): "tile128x128k256_mfma32"}.items():
        assert nv.nvfp4_gemm_epilogue_plan(M, N, K) == plan, (M, N, K)
    # one split, its counters, or partials of S tiles behind 4096 bytes of counters
    assert nv.nvfp4_gemm_epilogue_workspace_size(333, 2001, 1536) == 0
    assert nv.nvfp4_gemm_epilogue_workspace_size(1024, 768, 6144) == 4096 + 192 * 4 * 64 * 64 * 4
    assert nv.nvfp4_gemm_gated_plan(1, 2048, 6144).startswith("gatedreg16x8")
    assert nv.nvfp4_gemm_gated_plan(8192, 8192, 6144).startswith("gated256x128")
    for f in (nv.nvfp4_gemm_epilogue_plan, nv.nvfp4_gemm_gated_plan):
        assert f(16, 16, 100) == "none" and f(0, 16, 256) == "none" and f(1 << 22, 1 << 22, 256) == "none" and f(1 << 30, 32, 256) == "none"
    assert nv.nvfp4_gemm_gated_workspace_size(-1, 16, 256) == 0




def test_binding_refuses_host_tensors():
    import torch
    t = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(nv.Nvfp4Error) as e:
        nv.nvfp4_residual_norm(t, None, None, None, 0, None, 1.0, None, None, 1e-6, 0, None, t, None, None, None, 4, 64)
    assert e.value.status == NULL and "GPU tensor" in str(e.value)
    with pytest.raises(nv.Nvfp4Error):
        nv.nvfp4_gemm_gated(t, t, t, t, None, None, 0, t, 4, 64, 256)
