"""The mixture-of-experts operators where byte offsets, element counts or row
counts pass 2^31 and 2^32: the last and some other rows against the oracle."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_07_amd as nv
from oracle import experts_ref as x
from oracle import mxfp4_ref as mx
from tests.experts_util import U, dev_mx, mx_operand, offsets_of, product_bound
from tests.gpu_util import dev, host, say

pytestmark = pytest.mark.gpu


def codes(g, *shape):
    return torch.randint(0, 256, shape, dtype=torch.uint8, device="cuda", generator=g)


def scales(g, *shape):
    return torch.randint(122, 131, shape, dtype=torch.uint8, device="cuda", generator=g)


def products(a, a_sf, b, b_sf):
    A, B = mx.dequant(a, a_sf), mx.dequant(b, b_sf)
    return A @ B.T, np.abs(A) @ np.abs(B).T


@pytest.mark.parametrize("E,rows", [(5000, 300000), (3, 300000)])  # 64-row tiles and weights of 5 GB; 256-row tiles
def test_outputs_and_weights_above_4_gib(E, rows):
    N, K = 8200, 256
    say("large outputs", E, rows, N, K)
    g = torch.Generator(device="cuda").manual_seed(E)
    a, a_sf, b, b_sf = codes(g, rows, K // 2), scales(g, rows, K // 32), codes(g, E, N, K // 2), scales(g, E, N, K // 32)
    d = torch.full((rows, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    off = offsets_of([rows // E] * E)
    nv.nvfp4_mx_grouped_gemm(a, a_sf, None, b, b_sf, dev(off), None, None, d, rows, rows, N, K, E)
    assert d.numel() * 2 > 2 ** 32 and not bool(torch.isnan(d).any())
    for e in (0, E // 2, E - 1):
        at = slice(int(off[e + 1]) - 20, int(off[e + 1]))
        s, mag = products(host(a[at]), host(a_sf[at]), host(b[e]), host(b_sf[e]))
        assert (np.abs(host(d[at].double()) - s) <= product_bound(s, mag, K)).all()


@pytest.mark.parametrize("counts", [[9, 31], [200, 201]])
def test_tokens_up_to_2_31_bytes(counts):
    K, N = 4096, 96
    T, E, rows = (2 ** 32 - 1) // K, len(counts), sum(counts)
    say("many tokens", T, K, counts)
    g = torch.Generator(device="cuda").manual_seed(1)
    a, a_sf = codes(g, T, K // 2), scales(g, T, K // 32)
    b, b_sf = mx_operand(5, E, N, K)
    tok = np.random.default_rng(2).integers(0, T, rows).astype(np.int32)
    tok[::3] = T - 1 - np.arange(tok[::3].size)
    tok[1::17] = T  # outside
    d = torch.full((rows, N), float("nan"), dtype=torch.bfloat16, device="cuda")
    off = offsets_of(counts)
    nv.nvfp4_mx_grouped_gemm(a, a_sf, dev(tok), *dev_mx(b, b_sf), dev(off), None, None, d, rows, T, N, K, E)
    at = torch.from_numpy(np.minimum(tok, T - 1).astype(np.int64)).cuda()
    s, mag = x.expert_products(host(a[at]), host(a_sf[at]), np.where(tok < T, np.arange(rows), -1), b, b_sf, off, rows)
    assert (np.abs(host(d.double()) - s) <= product_bound(s, mag, K)).all()
    assert (host(d.float())[1::17] == 0).all()


def test_quantisation_of_more_than_2_32_elements():
    R, K = 66000, 65536
    say("large quantisation", R, K)
    rng = np.random.default_rng(3)
    some = np.array([0, 32767, 32768, R - 1])
    v = torch.from_numpy(rng.standard_normal((4, K)).astype(np.float32)).bfloat16()
    v32 = v.float().numpy()
    want = x.quantize(v32, x.FLOOR)
    at = torch.from_numpy(some).cuda()

    def check(q, sf, rows=some):
        at = torch.from_numpy(rows).cuda()
        np.testing.assert_array_equal(host(q[at]), want[0])
        np.testing.assert_array_equal(host(sf[at]), want[1])
        assert not bool(q[1:32767].any()) and not bool(sf[1:32767].any()) and not bool(q[32769:R - 1].any())
    q, sf = torch.empty(R, K // 2, dtype=torch.uint8, device="cuda"), torch.empty(R, K // 32, dtype=torch.uint8, device="cuda")
    wide = torch.zeros(R, K, device="cuda")
    wide[at] = v.float().cuda()
    nv.nvfp4_mx_quantize(wide, R, K, nv.MX_FLOOR, q, sf)
    check(q, sf)
    del wide
    half = torch.zeros(R, K, dtype=torch.bfloat16, device="cuda")
    half[at] = v.cuda()
    q.fill_(0x77)
    nv.nvfp4_mx_quantize_rows_bf16(half, None, nv.MX_FLOOR, q, sf, R, R, K)
    check(q, sf)
    q.fill_(0x77)
    back = torch.arange(R - 1, -1, -1, dtype=torch.int32, device="cuda")
    nv.nvfp4_mx_quantize_rows_bf16(half, back, nv.MX_FLOOR, q, sf, R, R, K)
    at = torch.from_numpy(R - 1 - some).cuda()
    np.testing.assert_array_equal(host(q[at]), want[0])
    np.testing.assert_array_equal(host(sf[at]), want[1])


def test_routing_of_more_than_2_32_logits():
    T, E, k = 2 ** 22 + 5, 1024, 8
    say("many logits", T, E, k)
    g = torch.Generator(device="cuda").manual_seed(4)
    logits = torch.empty(T, E, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    bias = torch.randn(E, device="cuda", generator=g) * 0.01
    ids, w = torch.full((T, k), -7, dtype=torch.int32, device="cuda"), torch.full((T, k), -7.0, device="cuda")
    nv.nvfp4_moe_route(logits, bias, nv.SCORE_SIGMOID, 8, 4, 2, k, True, 1.0, ids, w, T, E)
    assert int(ids.min()) >= 0 and int(ids.max()) < E
    at = torch.tensor([0, 1, T // 2, T - 2, T - 1], device="cuda")
    want, ww = x.route(host(logits[at].float()), host(bias), x.SIGMOID, 8, 4, 2, k, True, 1.0)
    np.testing.assert_array_equal(host(ids[at]), want)
    assert (np.abs(host(w[at]) - ww) <= 24 * U * ww).all()  # 22 units, and the scale's product


def test_row_order_of_2_30_ids():
    T, E, k = 2 ** 27, 16, 8
    n = T * k
    say("row order of", n, "ids")
    g = torch.Generator(device="cuda").manual_seed(5)
    ids = torch.randint(-1, E, (n,), dtype=torch.int32, device="cuda", generator=g)  # some are left out
    ids[n - 5 * 32768:] = 3  # runs of one expert
    i32 = lambda n: torch.full((n,), -7, dtype=torch.int32, device="cuda")
    off, tok, rows = i32(E + 1), i32(n), i32(n)
    nv.nvfp4_moe_sort(ids, 0, off, tok, rows, T, E, k, nv.moe_sort_workspace(T, E, k))
    counts = [int((ids == e).sum()) for e in range(E)]
    np.testing.assert_array_equal(host(off), offsets_of(counts))
    next_row = host(off)[:E].astype(np.int64)
    part = 2 ** 26
    for lo in range(0, n, part):
        i, r = ids[lo:lo + part], rows[lo:lo + part]
        for e in range(E):  # the expert's rows in this part follow those before
            mine = r[i == e]
            assert torch.equal(mine, torch.arange(next_row[e], next_row[e] + mine.numel(), dtype=torch.int32, device="cuda"))
            next_row[e] += mine.numel()
        assert bool((r[i < 0] == -1).all())
        there = torch.nonzero(i >= 0).flatten()
        assert torch.equal(tok[r[there].long()].long(), (there + lo) // k)
    assert bool((tok[sum(counts):] == -7).all())
