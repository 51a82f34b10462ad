"""The grouped MXFP4 products against the fp64 oracle."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_07_amd as nv
from oracle import experts_ref as x
from tests.experts_util import U, check_mx, dev_mx, mx_operand, offsets_of, out_bytes, product_bound
from tests.gpu_util import dev, host, say

pytestmark = pytest.mark.gpu
FILL = 0x7FC1  # a NaN that no product gives

COUNTS = {
    "one row": [1],
    "empty among them": [0, 3, 0, 0, 17, 1, 0],
    "one has all": [0, 0, 70, 0],
    "around the tiles": [15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65],
    "more than a tile": [129, 2, 200],
    "many": [300, 0, 513, 1, 260],
}


def problem(seed, counts, N, K, gather, T=None):
    E, rows = len(counts), int(np.sum(counts))
    rng = np.random.default_rng(seed)
    T = (max(1, rows // 3) if gather else rows) if T is None else T
    a, a_sf = mx_operand(seed, T, K)
    b, b_sf = mx_operand(seed + 10, E, N, K)
    tok = rng.integers(0, T, rows).astype(np.int32) if gather else None
    return dict(a=a, a_sf=a_sf, tok=tok, b=b, b_sf=b_sf, off=offsets_of(counts), E=E, rows=rows, T=T, N=N, K=K)


def expert_of(p):
    return np.repeat(np.arange(p["E"]), np.diff(p["off"]))


def gemm(p, alpha=None, bias=None, rows=None, status=None):
    a, a_sf, b, b_sf = dev_mx(p["a"], p["a_sf"], p["b"], p["b_sf"])
    rows = p["rows"] if rows is None else rows
    d = torch.full((rows, p["N"]), FILL, dtype=torch.int16, device="cuda").view(torch.bfloat16)
    nv.nvfp4_mx_grouped_gemm(a, a_sf, None if p["tok"] is None else dev(p["tok"]), b, b_sf, dev(p["off"]),
                             None if alpha is None else dev(alpha), None if bias is None else dev(bias).bfloat16(), d, rows,
                             p["T"], p["N"], p["K"], p["E"], status)
    return d


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("N,K", [(1, 256), (64, 512), (129, 768), (200, 1024), (333, 1280), (256, 2304)])
@pytest.mark.parametrize("name", list(COUNTS))
def test_gemm(name, N, K, gather):
    say("mx grouped", name, N, K, gather)
    p = problem(N + K, COUNTS[name], N, K, gather)
    s, mag = x.expert_products(p["a"], p["a_sf"], p["tok"], p["b"], p["b_sf"], p["off"], p["rows"])
    got = gemm(p).double().cpu().numpy()
    assert (np.abs(got - s) <= product_bound(s, mag, K)).all()
    e = expert_of(p)
    rng = np.random.default_rng(1)
    alpha = rng.uniform(0.5, 2, p["E"]).astype(np.float32)
    bias = torch.from_numpy(rng.standard_normal((p["E"], N)).astype(np.float32) * 50).bfloat16().float().numpy()
    got = gemm(p, alpha, bias).double().cpu().numpy()
    al, bi = alpha[e].astype(np.float64)[:, None], bias[e].astype(np.float64)
    assert (np.abs(got - (al * s + bi)) <= product_bound(s, mag, K, al, bi)).all()


@pytest.mark.parametrize("act", [0, 1, 2, 3, 4])
@pytest.mark.parametrize("rule", [nv.MX_FLOOR, nv.MX_CEIL])
@pytest.mark.parametrize("name,I,K,gather", [("one row", 32, 256, False), ("empty among them", 96, 512, True),
                                             ("around the tiles", 160, 1280, True), ("more than a tile", 64, 768, False),
                                             ("many", 288, 1024, True)])
def test_gated(name, I, K, gather, rule, act):
    say("mx gated", name, I, K, gather, rule, act)
    p = problem(I + K, COUNTS[name], 2 * I, K, gather)
    p["a_sf"] = (p["a_sf"].astype(np.int64) - 7).astype(np.uint8)  # gates of a few units
    p["b_sf"] = (p["b_sf"].astype(np.int64) - 5).astype(np.uint8)
    e = expert_of(p)
    rng = np.random.default_rng(2)
    alpha = rng.uniform(0.5, 2, 2 * p["E"]).astype(np.float32)
    bias = torch.from_numpy(rng.standard_normal((p["E"], 2 * I)).astype(np.float32)).bfloat16().float().numpy()
    s, mag = x.expert_products(p["a"], p["a_sf"], p["tok"], p["b"], p["b_sf"], p["off"], p["rows"])
    a, a_sf, b, b_sf = dev_mx(p["a"], p["a_sf"], p["b"], p["b_sf"])
    for al, bi in ((None, None), (alpha, bias)):
        q, sf = out_bytes(p["rows"], I, 2), out_bytes(p["rows"], I, 32)
        nv.nvfp4_mx_grouped_gated_quantize(a, a_sf, None if p["tok"] is None else dev(p["tok"]), b, b_sf, dev(p["off"]),
                                           None if al is None else dev(al), None if bi is None else dev(bi).bfloat16(), act,
                                           rule, q, sf, p["rows"], p["T"], I, K, p["E"])
        a0, a1 = (np.ones(2 * p["E"]) if al is None else al.astype(np.float64)).reshape(-1, 2)[e].T[..., None]
        bb = np.zeros((p["E"], 2 * I)) if bi is None else bi.astype(np.float64)
        g, u = a0 * s[:, :I] + bb[e][:, :I], a1 * s[:, I:] + bb[e][:, I:]
        # errors of both factors (fp32 sums of K products, a product, a sum), through act (slope at
        # most 1.13) and the product; act and the product themselves within 64 U
        dg, du = (np.abs(f) * (K + 3) * U * m + 2 * U * np.abs(v) for f, m, v in ((a0, mag[:, :I], g), (a1, mag[:, I:], u)))
        f = x.activation(g, act)
        h = f * u
        delta = 1.13 * dg * (np.abs(u) + du) + np.abs(f) * du + 64 * U * np.abs(h) + 2.0 ** -140
        # an activation's own error is relative to its argument where it vanishes
        delta += 64 * U * np.minimum(np.abs(g), 1.0) * np.abs(u) * (act != 0)
        check_mx(host(q), host(sf), h, delta, rule, name)


def check_gemm(p, got, bias=None):
    s, mag = x.expert_products(p["a"], p["a_sf"], p["tok"], p["b"], p["b_sf"], p["off"], p["rows"])
    bi = 0.0 if bias is None else bias[expert_of(p)].astype(np.float64)
    assert (np.abs(got.double().cpu().numpy() - (s + bi)) <= product_bound(s, mag, p["K"], 1.0, bi)).all()


@pytest.mark.parametrize("K", [256, 768])
def test_more_tiles_than_work_groups(K):
    # 8 row tiles of 50 column tiles, the last of each in part: work-groups go through several
    p = problem(K, [700, 0, 300, 513], 12600, K, True)
    bias = torch.from_numpy(np.random.default_rng(3).standard_normal((4, 12600)).astype(np.float32) * 50).bfloat16().float().numpy()
    check_gemm(p, gemm(p, bias=bias), bias)
    p["a_sf"] = (p["a_sf"].astype(np.int64) - 7).astype(np.uint8)
    s, mag = x.expert_products(p["a"], p["a_sf"], p["tok"], p["b"], p["b_sf"], p["off"], p["rows"])
    I = 6272
    b, b_sf = (np.concatenate([v[:, :I], v[:, -I:]], 1) for v in (p["b"], p["b_sf"]))
    s, mag = (np.concatenate([v[:, :I], v[:, -I:]], 1) for v in (s, mag))
    a, a_sf, b, b_sf = dev_mx(p["a"], p["a_sf"], b, b_sf)
    q, sf = out_bytes(p["rows"], I, 2), out_bytes(p["rows"], I, 32)
    nv.nvfp4_mx_grouped_gated_quantize(a, a_sf, dev(p["tok"]), b, b_sf, dev(p["off"]), None, None, 0, 1, q, sf, p["rows"], p["T"],
                                       I, K, 4)
    (dg, g), (du, u) = (((K + 3) * U * m + 2 * U * np.abs(v), v) for m, v in ((mag[:, :I], s[:, :I]), (mag[:, I:], s[:, I:])))
    h = g * u
    check_mx(host(q), host(sf), h, dg * (np.abs(u) + du) + np.abs(g) * du + 4 * U * np.abs(h) + 2.0 ** -140, 1, "persistent")


@pytest.mark.parametrize("E,counts", [(300, {0: 3, 3: 1, 255: 17, 256: 2, 299: 40}), (300, {7: 22000, 280: 90}), (1100, {1099: 70, 64: 1}),
                                      (1100, {1030: 79300})])
def test_many_experts(E, counts):
    say("experts", E, counts)
    n = [counts.get(e, 0) for e in range(E)]
    check_gemm(*(lambda p: (p, gemm(p)))(problem(E, n, 40, 256, True, T=50)))


@pytest.mark.parametrize("rows,N", [(64, 64), (2000, 64), (2000, 300)])
def test_offsets_that_go_back_and_forth(rows, N):
    # every other expert claims all rows: it ends, and whole rows come out
    E = 16
    p = problem(rows, [rows] + [0] * (E - 1), N, 256, True)
    p["off"] = np.array([0, rows] * (E // 2) + [0], np.int32)
    status = torch.full((1,), -9, dtype=torch.int32, device="cuda")
    p["b"][:], p["b_sf"][:] = p["b"][0], p["b_sf"][0]  # whichever writes a row
    got = gemm(p, status=status)
    assert host(status)[0] == 2
    p["off"] = offsets_of([rows] + [0] * (E - 1))
    s, mag = x.expert_products(p["a"], p["a_sf"], p["tok"], p["b"], p["b_sf"], p["off"], rows)
    near = np.abs(got.double().cpu().numpy() - s) <= product_bound(s, mag, 256)
    assert (near | (host(got.view(torch.int16)) == FILL)).all() and near.any()


def test_rows_behind_the_last_expert_stay():
    p = problem(5, [3, 0, 9], 100, 512, True)
    p["tok"] = np.concatenate([p["tok"], np.full(20, 2 ** 30, np.int32)])  # never read
    status = torch.full((1,), -9, dtype=torch.int32, device="cuda")
    d = gemm(p, rows=32, status=status)
    assert (host(d.view(torch.int16))[12:] == FILL).all() and host(status)[0] == 0
    assert not (host(d.view(torch.int16))[:12] == FILL).any()
    a, a_sf, b, b_sf = dev_mx(p["a"], p["a_sf"], p["b"][:, :64], p["b_sf"][:, :64])
    q, sf = out_bytes(32, 32, 2), out_bytes(32, 32, 32)
    nv.nvfp4_mx_grouped_gated_quantize(a, a_sf, dev(p["tok"]), b, b_sf, dev(p["off"]), None, None, 4, 0, q, sf, 32, p["T"], 32,
                                       512, 3)
    assert (host(q)[12:] == 0xA5).all() and (host(sf)[12:] == 0xA5).all()


@pytest.mark.parametrize("off,bad", [([0, 5, 3, 8], 2), ([0, 4, 99, 99], 2), ([-1, 4, 5, 8], 1), ([0, 2, 2, 8], 0), ([0, 8, 8, 8], 0)])
def test_status_of_offsets(off, bad):
    p = problem(6, [2, 3, 3], 64, 256, False)
    p["off"] = np.array(off, np.int32)
    status = torch.full((1,), -9, dtype=torch.int32, device="cuda")
    got = host(gemm(p, status=status).view(torch.int16))
    assert host(status)[0] == bad
    good = [e for e in range(3) if 0 <= off[e] <= off[e + 1] <= 8]
    covered = np.zeros(8, bool)
    for e in good:
        covered[off[e]:off[e + 1]] = True
    assert ((got != FILL).all(1) == covered).all()


def test_tokens_outside_read_as_zero_rows():
    p = problem(7, [4, 4], 64, 512, True, T=5)
    p["tok"] = np.array([0, -1, 4, 5, 2 ** 31 - 1, 1, -2 ** 31, 2], np.int32)
    status = torch.full((1,), -9, dtype=torch.int32, device="cuda")
    bias = np.ones((2, 64), np.float32)
    got = gemm(p, bias=bias, status=status).double().cpu().numpy()
    assert host(status)[0] == -2
    assert (got[[1, 3, 4, 6]] == 1.0).all()
    s, mag = x.expert_products(p["a"], p["a_sf"], p["tok"], p["b"], p["b_sf"], p["off"], 8)
    assert (np.abs(got - (s + 1)) <= product_bound(s, mag, 512, 1.0, 1.0)).all()


def test_nan_scales_reach_what_reads_them():
    p = problem(8, [3, 20], 96, 768, False)
    p["a_sf"][1, 5] = 0xFF      # row 1
    p["a"][1, 80:96] = 0        # its codes are zeros, as the quantisation leaves them
    p["b_sf"][1, 40, 0] = 0xFF  # column 40 of expert 1
    got = gemm(p).double().cpu().numpy()
    nan = np.zeros((23, 96), bool)
    nan[1], nan[3:, 40] = True, True
    assert (np.isnan(got) == nan).all()
    a, a_sf, b, b_sf = dev_mx(p["a"], p["a_sf"], p["b"][:, :64], p["b_sf"][:, :64])
    q, sf = out_bytes(23, 32, 2), out_bytes(23, 32, 32)
    nv.nvfp4_mx_grouped_gated_quantize(a, a_sf, None, b, b_sf, dev(p["off"]), None, None, 4, 0, q, sf, 23, 23, 32, 768, 2)
    nan = np.zeros(23, bool)
    nan[1], nan[3:] = True, True
    assert ((host(sf)[:, 0] == 0xFF) == nan).all() and (host(q)[nan] == 0).all()


def test_odd_addresses():
    # outputs and bias at odd 2-byte addresses, and a row length that is no multiple of 4
    p = problem(9, [5, 18], 77, 256, False)
    want = host(gemm(p, bias=np.full((2, 77), 2.0, np.float32)).view(torch.int16))
    a, a_sf, b, b_sf = dev_mx(p["a"], p["a_sf"], p["b"], p["b_sf"])
    room = torch.full((23 * 77 + 2,), FILL, dtype=torch.int16, device="cuda")
    bias = torch.full((2 * 77 + 1,), 2.0, dtype=torch.bfloat16, device="cuda")[1:]
    nv.nvfp4_mx_grouped_gemm(a, a_sf, None, b, b_sf, dev(p["off"]), None, bias, room[1:-1], 23, 23, 77, 256, 2)
    np.testing.assert_array_equal(host(room)[1:-1].reshape(23, 77), want)
    assert host(room)[0] == FILL and host(room)[-1] == FILL


def test_nothing_to_do():
    p = problem(10, [2], 64, 256, False)
    a, a_sf, b, b_sf = dev_mx(p["a"], p["a_sf"], p["b"], p["b_sf"])
    off = dev(np.zeros(2, np.int32))
    status = torch.full((1,), -9, dtype=torch.int32, device="cuda")
    nv.nvfp4_mx_grouped_gemm(None, None, None, b, b_sf, off, None, None, None, 0, 0, 64, 256, 1, status)
    assert host(status)[0] == 0
    d = torch.full((2, 64), FILL, dtype=torch.int16, device="cuda")
    nv.nvfp4_mx_grouped_gemm(a, a_sf, None, b, b_sf, off, None, None, d, 2, 2, 64, 256, 1)  # no expert has rows
    assert (host(d) == FILL).all()


def test_refused_tensors():
    p = problem(11, [4, 4], 64, 256, True, T=4)
    a, a_sf, b, b_sf = dev_mx(p["a"], p["a_sf"], p["b"], p["b_sf"])
    tok, off, d = dev(p["tok"]), dev(p["off"]), torch.empty(8, 64, dtype=torch.bfloat16, device="cuda")

    def call(**kw):
        t = dict(a=a, a_sf=a_sf, row_token=tok, b=b, b_sf=b_sf, offsets=off, alpha=None, bias=None, d=d, rows=8, T=4, N=64, K=256,
                 E=2)
        t.update(kw)
        return nv.nvfp4_mx_grouped_gemm(**t)
    call()
    for bad in (dict(a=a[:3]), dict(a_sf=a_sf[:, :7]), dict(row_token=tok[:7]), dict(row_token=tok.long()), dict(b=b[:1]),
                dict(b_sf=b_sf[:1]), dict(offsets=off[:2]), dict(offsets=off.long()), dict(alpha=torch.ones(1, device="cuda")),
                dict(bias=torch.ones(1, 64, dtype=torch.bfloat16, device="cuda")), dict(d=d[:7]), dict(d=d.float()),
                dict(row_token=None), dict(E=3), dict(K=512), dict(N=65), dict(a=a.cpu())):
        with pytest.raises(nv.Nvfp4Error):
            call(**bad)
