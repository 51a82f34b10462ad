"""Host-side refusals, sizes and no-ops of the mixture-of-experts operators (CPU
only: every call is answered before any HIP call)."""
import pytest

import nvfp4_block_scaled_07_amd as nv

FAKE = 0x10000  # an aligned non-NULL address; never dereferenced
NULL, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5


def _call(fn, defaults, kw):
    args = {**defaults, **kw}
    assert set(args) == set(defaults)
    return getattr(nv.lib(), fn)(*args.values())


def _route(**kw):
    return _call("nvfp4_moe_route", dict(logits=FAKE, type=0, ldl=0, bias=None, score=0, n_group=1, topk_group=1,
                                         group_top=1, top_k=2, renormalize=1, scale=1.0, ids=FAKE, weights=FAKE, T=4,
                                         E=8, stream=None), kw)


def _sort(**kw):
    return _call("nvfp4_moe_sort", dict(ids=FAKE, first=0, offsets=FAKE, row_token=FAKE, token_rows=FAKE, T=4, E=8,
                                        top_k=2, ws=None, wsb=0, stream=None), kw)


def _quant(**kw):
    return _call("nvfp4_mx_quantize", dict(x=FAKE, R=4, K=64, rule=0, q=FAKE, sf=FAKE, stream=None), kw)


def _rows(**kw):
    return _call("nvfp4_mx_quantize_rows_bf16", dict(x=FAKE, tok=None, rule=0, q=FAKE, sf=FAKE, rows=4, T=4, K=64,
                                                     stream=None), kw)


def _gemm(**kw):
    return _call("nvfp4_mx_grouped_gemm", dict(a=FAKE, a_sf=FAKE, tok=FAKE, b=FAKE, b_sf=FAKE, offsets=FAKE, alpha=None,
                                               bias=None, d=FAKE, rows=8, T=4, N=16, K=256, E=4, status=None,
                                               stream=None), kw)


def _gated(**kw):
    return _call("nvfp4_mx_grouped_gated_quantize",
                 dict(a=FAKE, a_sf=FAKE, tok=FAKE, b=FAKE, b_sf=FAKE, offsets=FAKE, alpha=None, bias=None, act=4, rule=0,
                      q=FAKE, sf=FAKE, rows=8, T=4, N=64, K=256, E=4, status=None, stream=None), kw)


def _ffn(**kw):
    return _call("nvfp4_mx_moe_ffn", dict(x=FAKE, tok=FAKE, offsets=FAKE, gu=FAKE, gu_sf=FAKE, al=None, bg=None, act=4,
                                          rule=0, dn=FAKE, dn_sf=FAKE, ald=None, bd=None, tr=FAKE, tw=FAKE, out=FAKE,
                                          T=4, H=256, I=256, E=4, top_k=2, ws=FAKE, wsb=0, status=None, stream=None), kw)


def test_route_refusals():
    assert _route(T=-1) == SHAPE and _route(E=0) == SHAPE and _route(top_k=0) == SHAPE
    assert _route(type=2) == SHAPE and _route(score=2) == SHAPE and _route(score=-1) == SHAPE
    assert _route(n_group=3) == SHAPE and "n_group" in nv.nvfp4_last_error()
    assert _route(n_group=0) == SHAPE and _route(topk_group=2) == SHAPE and _route(topk_group=0) == SHAPE
    assert _route(group_top=3) == SHAPE and _route(group_top=0) == SHAPE
    assert _route(top_k=9) == SHAPE and _route(n_group=4, topk_group=2, top_k=5) == SHAPE
    assert _route(ldl=7) == SHAPE and "ldl" in nv.nvfp4_last_error()
    assert _route(E=1025) == UNSUPPORTED and _route(E=128, top_k=65) == UNSUPPORTED
    assert _route(E=128, n_group=128, topk_group=128) == UNSUPPORTED and _route(T=1 << 31) == UNSUPPORTED
    for name in ("logits", "ids", "weights"):
        assert _route(**{name: None}) == NULL and _route(**{name: FAKE + 2}) == ALIGN
    assert _route(bias=FAKE + 2) == ALIGN and _route(type=1, logits=FAKE + 1) == ALIGN
    assert _route(T=0, logits=None, ids=None) == 0 and nv.nvfp4_last_error() == ""


def test_sort_refusals():
    assert _sort(T=-1) == SHAPE and _sort(E=0) == SHAPE and _sort(top_k=-1) == SHAPE and _sort(first=-1) == SHAPE
    assert _sort(E=65536) == UNSUPPORTED and _sort(T=1 << 30) == UNSUPPORTED and _sort(T=1 << 62) == UNSUPPORTED
    assert _sort(T=1 << 18, E=1025, top_k=5) == UNSUPPORTED and "1024" in nv.nvfp4_last_error()
    assert _sort(T=1 << 18, E=1025, top_k=4, ids=None) == NULL
    for name in ("ids", "offsets", "row_token", "token_rows"):
        assert _sort(**{name: None}) == NULL and _sort(**{name: FAKE + 2}) == ALIGN
    assert nv.nvfp4_moe_sort_workspace_size(-1, 8, 2) == 0 and nv.nvfp4_moe_sort_workspace_size(4, 0, 2) == 0
    assert nv.nvfp4_moe_sort_workspace_size(1 << 62, 8, 8) == 0
    need = nv.nvfp4_moe_sort_workspace_size(1 << 20, 256, 8)
    if need:
        big = dict(T=1 << 20, E=256, top_k=8)
        assert _sort(**big) == WORKSPACE and _sort(**big, ws=FAKE, wsb=need - 1) == WORKSPACE
        assert _sort(**big, ws=FAKE + 16, wsb=need) == ALIGN


def test_quantise_refusals():
    assert _quant(R=-1) == SHAPE and _quant(K=48) == SHAPE and "block size 32" in nv.nvfp4_last_error()
    assert _quant(K=-32) == SHAPE and _quant(rule=2) == SHAPE and _quant(rule=-1) == SHAPE
    assert _quant(K=(1 << 30) + 32) == UNSUPPORTED and _quant(R=1 << 60) == UNSUPPORTED
    assert _quant(x=None) == NULL and _quant(q=None) == NULL and _quant(sf=None) == NULL
    assert _quant(x=FAKE + 8) == ALIGN and _quant(q=FAKE + 8) == ALIGN
    assert _quant(R=0, x=None) == 0 and _quant(K=0, q=None) == 0
    assert _rows(rows=-1) == SHAPE and _rows(T=-1) == SHAPE and _rows(K=16) == SHAPE and _rows(rule=7) == SHAPE
    assert _rows(rows=5) == SHAPE and "row_token" in nv.nvfp4_last_error()
    assert _rows(rows=1 << 60, tok=FAKE) == UNSUPPORTED
    assert _rows(x=None) == NULL and _rows(q=None) == NULL and _rows(sf=None) == NULL
    assert _rows(x=FAKE + 2) == ALIGN and _rows(tok=FAKE + 2) == ALIGN
    assert _rows(rows=0, x=None) == 0


@pytest.mark.parametrize("call", [_gemm, _gated])
def test_product_refusals(call):
    for name in ("rows", "T", "N", "E"):
        assert call(**{name: -32}) == SHAPE
    assert call(K=40) == SHAPE and "block size 32" in nv.nvfp4_last_error()
    assert call(K=128) == UNSUPPORTED and call(K=0) == UNSUPPORTED and call(K=(1 << 22) + 256) == UNSUPPORTED
    assert call(tok=None) == SHAPE and "row_token" in nv.nvfp4_last_error()
    assert call(T=1 << 24) == UNSUPPORTED and "T K" in nv.nvfp4_last_error()
    assert call(T=1 << 62) == UNSUPPORTED and call(rows=1 << 31) == UNSUPPORTED and call(N=1 << 31) == UNSUPPORTED
    assert call(E=65536) == UNSUPPORTED and call(E=65535, N=1 << 20, rows=1 << 20) == UNSUPPORTED
    for name in ("a", "a_sf", "b", "b_sf"):
        assert call(**{name: None}) == NULL and call(**{name: FAKE + 8}) == ALIGN
    assert call(offsets=None) == NULL
    for name in ("offsets", "tok", "alpha", "status"):
        assert call(**{name: FAKE + 2}) == ALIGN
    assert call(bias=FAKE + 1) == ALIGN
    assert call(rows=0, a=None) == 0 and call(N=0, b=None) == 0 and call(E=0, offsets=None) == 0
    assert nv.nvfp4_last_error() == ""


def test_output_refusals():
    assert _gemm(d=None) == NULL and _gemm(d=FAKE + 1) == ALIGN
    assert _gated(q=None) == NULL and _gated(sf=None) == NULL and _gated(q=FAKE + 1) == ALIGN
    assert _gated(N=48) == SHAPE and _gated(act=5) == SHAPE and _gated(act=-1) == SHAPE and _gated(rule=2) == SHAPE


def test_ffn_refusals():
    need = nv.nvfp4_mx_moe_ffn_workspace_size(4, 256, 256, 2)
    assert need > 0
    ok = dict(wsb=need)
    assert _ffn() == WORKSPACE and _ffn(ws=None, wsb=need) == WORKSPACE and _ffn(wsb=need - 1) == WORKSPACE
    assert _ffn(ws=FAKE + 16, **ok) == ALIGN
    assert _ffn(T=-1, **ok) == SHAPE and _ffn(E=-1, **ok) == SHAPE and _ffn(top_k=-1, **ok) == SHAPE
    assert _ffn(H=264, **ok) == SHAPE and _ffn(I=128, **ok) == UNSUPPORTED and _ffn(H=128, **ok) == UNSUPPORTED
    assert _ffn(E=0, **ok) == SHAPE and _ffn(act=9, **ok) == SHAPE and _ffn(rule=3, **ok) == SHAPE
    assert _ffn(T=1 << 25, **ok) == UNSUPPORTED and _ffn(T=1 << 62, **ok) == UNSUPPORTED
    for name in ("x", "out", "tok", "tr", "tw", "offsets", "gu", "gu_sf", "dn", "dn_sf"):
        assert _ffn(**{name: None}, **ok) == NULL, name
        assert _ffn(**{name: FAKE + 2}, **ok) == ALIGN, name
    for name in ("al", "ald", "status"):
        assert _ffn(**{name: FAKE + 2}, **ok) == ALIGN
    for name in ("bg", "bd"):
        assert _ffn(**{name: FAKE + 1}, **ok) == ALIGN
    assert _ffn(T=0, x=None, ws=None) == 0
    size = nv.nvfp4_mx_moe_ffn_workspace_size
    assert size(-1, 256, 256, 2) == 0 and size(4, 128, 256, 2) == 0 and size(1 << 62, 256, 256, 8) == 0
