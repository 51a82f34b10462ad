"""nvfp4_residual_norm on the GPU through the C ABI: r, y and the NVFP4 codes
and scales bit for bit against the same steps in numpy (oracle.block_ref), and
against the formulas in fp64; every row length class, odd lengths, strides,
gates, in-place outputs, extreme values."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_07_amd as nv
from oracle import block_ref as br
from oracle import nvfp4_ref as o
from tests.block_util import bf16, dev_bf16, values
from tests.gpu_util import bits, host, say, scalar

pytestmark = pytest.mark.gpu

EPS = 1e-6


def _case(T, H, seed, kind, post, gate_group, residual):
    rng = np.random.default_rng(seed)
    vec = lambda m, s: bf16(rng.standard_normal(H) * s + m)
    layer = kind == nv.NORM_LAYER
    rows = 0 if gate_group is None else 1 if gate_group == 0 else -(-T // gate_group)
    return dict(x=bf16(rng.standard_normal((T, H)) * 2 + 0.25),
                post_w=vec(1, 0.2) if post else None, post_b=vec(0, 0.1) if post and layer else None,
                gate=bf16(rng.standard_normal((rows, H)) * 0.3 + 0.7) if rows else None, gate_group=gate_group or 0,
                res=bf16(rng.standard_normal((T, H)) * 3) if residual else None, beta=0.75 if residual else 1.0,
                w=vec(1, 0.2), b=vec(0, 0.1) if layer else None, eps=EPS, kind=kind)


def _opt(v):
    return None if v is None else dev_bf16(v)


def _run(c, T, H, r, y, gs=None, q=None, sf=None, x=None, res=None):
    return nv.nvfp4_residual_norm(_opt(c["x"]) if x is None else x, _opt(c["post_w"]), _opt(c["post_b"]), _opt(c["gate"]),
                                  c["gate_group"], _opt(c["res"]) if res is None else res, c["beta"], _opt(c["w"]),
                                  _opt(c["b"]), c["eps"], c["kind"], r, y, gs, q, sf, T, H)


def _new(T, H):
    return torch.full((T, H), 777.0, dtype=torch.bfloat16, device="cuda")


def _same_bits(t, want32, label):
    np.testing.assert_array_equal(bits(t.view(torch.int16)), o.bf16_rne(want32.astype(np.float64)), err_msg=label)


def _check(T, H, seed, kind, post, gate_group, residual):
    c = _case(T, H, seed, kind, post, gate_group, residual)
    say("norm", T, H, kind, post, gate_group, residual)
    r32, y32 = br.residual_norm(**c)
    r, y = _new(T, H), _new(T, H)
    quant = H % 16 == 0
    gs = np.float32(2688.0 / 6.0)
    q = torch.full((T, H // 2), 0xEE, dtype=torch.uint8, device="cuda") if quant else None
    sf = torch.full((T, H // 16), 0xEE, dtype=torch.uint8, device="cuda") if quant else None
    _run(c, T, H, r, y, scalar(gs) if quant else None, q, sf)
    _same_bits(r, r32, "r")
    _same_bits(y, y32, "y")
    if quant:
        rq, rsf = o.quantize(y32, gs)
        np.testing.assert_array_equal(host(sf), rsf)
        np.testing.assert_array_equal(host(q), rq)
    # the formulas: r and y within half a bf16 step and the fp32 steps' roundings.  Relative to each output's
    # terms: r has at most 6 steps; y adds rstd's rounding, the subtraction, two products and the bias, and the
    # second norm carries r's error to y (times at most 2 for the row's norm, which r's errors move too).
    re, ye = br.residual_norm_exact(**c)
    u = 2.0 ** -24
    big = np.abs(re).max(axis=1, keepdims=True) + (0 if c["res"] is None else 0.75 * np.abs(c["res"]).max())
    dr = 8 * u * big
    assert (np.abs(values(r) - re) <= 2.0 ** -8 * np.abs(re) + 2 * dr).all()
    scale = (np.abs(ye).max(axis=1, keepdims=True) + 1) / np.maximum(np.sqrt(((re - (re.mean(1, keepdims=True) if kind else 0)) ** 2).mean(1, keepdims=True)), 1e-3)
    assert (np.abs(values(y) - ye) <= 2.0 ** -8 * np.abs(ye) + 2 * (dr * scale * 4 + 16 * u * (np.abs(ye).max() + 1))).all()


# chunks of 8 columns per row: one thread group of each size, its last partial one, and rows past the registers
LENGTHS = [1, 7, 16, 48, 64, 512, 520, 1000, 1024, 1040, 1545, 2048, 2064, 4096, 4112, 6144, 6145, 8192, 8200, 12288,
           16384, 16400, 20011]


@pytest.mark.parametrize("H", LENGTHS)
@pytest.mark.parametrize("kind", [nv.NORM_RMS, nv.NORM_LAYER])
def test_lengths(H, kind):
    _check(5, H, H + kind, kind, True, None, True)


@pytest.mark.parametrize("H", [16, 1000, 1024, 1545, 2064, 4096, 6144, 6145, 8208, 12288, 12289, 16384])
@pytest.mark.parametrize("kind", [nv.NORM_RMS, nv.NORM_LAYER])
def test_many_rows(H, kind):
    # past two rows per CU the rows take fewer threads each
    _check(515, H, H + 7 * kind, kind, True, 100, True)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 37, 300])
@pytest.mark.parametrize("H", [96, 768, 6144])
def test_rows(T, H):
    _check(T, H, T + H, nv.NORM_RMS, False, None, True)


@pytest.mark.parametrize("kind", [nv.NORM_RMS, nv.NORM_LAYER])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate_group", [None, 0, 1, 5])
@pytest.mark.parametrize("residual", [False, True])
def test_combinations(kind, post, gate_group, residual):
    _check(13, 272, 7, kind, post, gate_group, residual)
    _check(6, 1545, 8, kind, post, gate_group, residual)


@pytest.mark.parametrize("H", [272, 1000, 20016])
def test_single_outputs(H):
    T = 9
    c = _case(T, H, 3, nv.NORM_RMS, True, 0, True)
    r32, y32 = br.residual_norm(**c)
    r = _new(T, H)
    _run(c, T, H, r, None)
    _same_bits(r, r32, "r alone")
    y = _new(T, H)
    _run(c, T, H, None, y)
    _same_bits(y, y32, "y alone")
    if H % 16 == 0:
        q = torch.zeros((T, H // 2), dtype=torch.uint8, device="cuda")
        sf = torch.zeros((T, H // 16), dtype=torch.uint8, device="cuda")
        _run(c, T, H, None, None, None, q, sf)
        rq, rsf = o.quantize(y32, np.float32(1.0))
        np.testing.assert_array_equal(host(sf), rsf)
        np.testing.assert_array_equal(host(q), rq)


@pytest.mark.parametrize("H", [272, 1545, 20016])
@pytest.mark.parametrize("into", ["x", "res"])
def test_r_in_place(H, into):
    T = 6
    c = _case(T, H, 5, nv.NORM_LAYER, True, 1, True)
    r32, y32 = br.residual_norm(**c)
    x, res, y = dev_bf16(c["x"]), dev_bf16(c["res"]), _new(T, H)
    _run(c, T, H, x if into == "x" else res, y, x=x, res=res)
    _same_bits(x if into == "x" else res, r32, "r in place")
    _same_bits(y, y32, "y")


@pytest.mark.parametrize("H,ld,off", [(272, 280, 0), (272, 275, 0), (272, 272, 1), (1545, 1600, 3), (20016, 20024, 0)])
def test_row_strides_offsets_and_padding(H, ld, off):
    T = 7
    c = _case(T, H, 6, nv.NORM_RMS, False, None, True)
    r32, y32 = br.residual_norm(**c)
    flats = [torch.full((T * ld + 8,), v, dtype=torch.bfloat16, device="cuda") for v in (float("nan"), float("nan"), -5.0, -5.0)]
    x, res, r, y = [f[off:off + T * ld].view(T, ld)[:, :H] for f in flats]
    x.copy_(dev_bf16(c["x"]))
    res.copy_(dev_bf16(c["res"]))
    _run(c, T, H, r, y, x=x, res=res)
    _same_bits(r.contiguous(), r32, "r")
    _same_bits(y.contiguous(), y32, "y")
    mask = np.ones(T * ld + 8, dtype=bool)
    mask[(off + np.arange(T)[:, None] * ld + np.arange(H)[None, :]).reshape(-1)] = False
    for f in flats[2:]:
        assert (host(f.float())[mask] == -5.0).all(), "padding was written"


@pytest.mark.parametrize("T,H", [((1 << 21) + 5, 4), ((1 << 21) + 3, 24)])
def test_more_rows_than_one_launch(T, H):
    # rows repeat with period 1001, so that a few of them stand for all
    c = _case(1001, H, 14, nv.NORM_LAYER, True, None, True)
    r32, y32 = br.residual_norm(**c)
    rows = torch.arange(T, device="cuda") % 1001
    x, res = dev_bf16(c["x"])[rows], dev_bf16(c["res"])[rows]
    r, y = _new(T, H), _new(T, H)
    _run(c, T, H, r, y, x=x, res=res)
    want = [dev_bf16(bf16(v))[rows] for v in (r32, y32)]
    assert torch.equal(r, want[0]) and torch.equal(y, want[1])


def test_a_gate_group_goes_on_over_launches():
    T, H, group = (1 << 21) + 700, 8, 1000
    c = _case(1, H, 15, nv.NORM_RMS, False, None, False)
    gate = torch.rand(-(-T // group), H, device="cuda").to(torch.bfloat16)
    x = torch.ones(T, H, device="cuda", dtype=torch.bfloat16)
    r = _new(T, H)
    nv.nvfp4_residual_norm(x, None, None, gate, group, None, 1.0, None, None, EPS, 0, r, None, None, None, None, T, H)
    assert torch.equal(r, gate.repeat_interleave(group, 0)[:T])


def test_rows_past_32_bit_offsets():
    # rows 2^30 + 8 elements apart: the last starts past 2^33 bytes
    T, H, ld = 5, 272, (1 << 30) + 8
    c = _case(T, H, 12, nv.NORM_RMS, True, None, True)
    r32, y32 = br.residual_norm(**c)
    big = torch.empty(4 * ld + 4 * H, dtype=torch.bfloat16, device="cuda")
    x, res, r, y = [big.as_strided((T, H), (ld, 1), i * H) for i in range(4)]
    x.copy_(dev_bf16(c["x"]))
    res.copy_(dev_bf16(c["res"]))
    _run(c, T, H, r, y, x=x, res=res)
    _same_bits(r.contiguous(), r32, "r")
    _same_bits(y.contiguous(), y32, "y")


@pytest.mark.parametrize("kind", [nv.NORM_RMS, nv.NORM_LAYER])
def test_zero_constant_and_large_rows(kind):
    # a zero row gives zeros (rstd = 1 / sqrt(eps)); a constant row has no variance; large values neither
    # overflow (the sums are fp64) nor lose the small rows beside them
    T, H = 6, 512
    c = _case(T, H, 9, kind, False, None, False)
    c["x"][0] = 0.0
    c["x"][1] = 3.0
    c["x"][2] *= bf16(np.float32(1e18))
    c["x"][3] *= 1e-18
    c["x"] = bf16(c["x"])
    r32, y32 = br.residual_norm(**c)
    assert np.isfinite(y32).all()
    y = _new(T, H)
    _run(c, T, H, None, y)
    _same_bits(y, y32, "y")


def test_non_finite_values_stay_in_their_row():
    T, H = 4, 768
    c = _case(T, H, 10, nv.NORM_RMS, True, None, True)
    c["x"][1, 5], c["res"][2, 7] = np.nan, np.inf
    r, y = _new(T, H), _new(T, H)
    _run(c, T, H, r, y)
    got_r, got_y = values(r), values(y)
    assert np.isnan(got_r[1]).all() and np.isnan(got_y[1]).all()
    # an infinite row norm: rstd is 0, and infinity times 0 is NaN
    assert got_r[2, 7] == np.inf and np.isnan(got_y[2, 7]) and (np.delete(got_y[2], 7) == 0).all()
    assert np.isfinite(got_y[[0, 3]]).all()


def test_graph_replays_and_streams():
    T, H = 40, 6144
    c = _case(T, H, 11, nv.NORM_RMS, True, 8, True)
    x, res = dev_bf16(c["x"]), dev_bf16(c["res"])
    vec = [_opt(c[k]) for k in ("post_w", "post_b", "gate")]
    w = _opt(c["w"])
    call = lambda r, y: nv.nvfp4_residual_norm(x, *vec, 8, res, 1.0, w, None, EPS, nv.NORM_RMS, r, y, None, None, None, T, H)
    r, y, r2, y2 = _new(T, H), _new(T, H), _new(T, H), _new(T, H)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(r2, y2)
    call(r, y)
    torch.cuda.synchronize()
    assert torch.equal(r, r2) and torch.equal(y, y2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(r2, y2)
    for i in range(4):
        x.mul_(-0.5)
        call(r, y)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(r, r2) and torch.equal(y, y2), f"replay {i}"
