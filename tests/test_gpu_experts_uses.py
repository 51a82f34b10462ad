"""Calls of the mixture-of-experts operators that their documentation allows and
that belong to no operator's own tests."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_07_amd as nv
from oracle import experts_ref as x
from oracle import moe_ref as m
from tests.experts_util import dev_mx, mx_operand, offsets_of, out_bytes
from tests.gpu_util import bits, dev, host, say, scalar
from tests.test_gpu_moe import _ffn_problem, _frob
from tests.test_gpu_moe_sort import fast

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts", [[3, 0, 5], [30, 41], [200, 300]])  # 16-, 64- and 256-row tiles
@pytest.mark.parametrize("K", [256, 2304])
def test_no_tokens_at_all(K, counts):
    # T == 0: every row's token is outside and reads as zeros
    say("no tokens", K, counts)
    E, rows, N = len(counts), sum(counts), 96
    b, b_sf = dev_mx(*mx_operand(K, E, N, K))
    a, a_sf = (torch.full((256,), v, dtype=torch.uint8, device="cuda") for v in (0x77, 0x80))  # never read
    tok = torch.zeros(rows, dtype=torch.int32, device="cuda")
    off = dev(offsets_of(counts))
    bias = torch.arange(E * N, device="cuda").reshape(E, N).bfloat16()
    status = torch.full((1,), -9, dtype=torch.int32, device="cuda")
    d = torch.full((rows, N), 7.0, dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_mx_grouped_gemm(a, a_sf, tok, b, b_sf, off, None, bias, d, rows, 0, N, K, E, status)
    want = host(bias.float())[np.repeat(np.arange(E), counts)]
    np.testing.assert_array_equal(host(d.float()), want)
    assert host(status)[0] == -1
    q, sf = out_bytes(rows, 32, 2), out_bytes(rows, 32, 32)
    nv.nvfp4_mx_grouped_gated_quantize(a, a_sf, tok, b[:, :64].contiguous(), b_sf[:, :64].contiguous(), off, None, None, 4, 0, q,
                                       sf, rows, 0, 32, K, E, status)
    assert (host(q) == 0).all() and (host(sf) == 0).all() and host(status)[0] == -1
    q, sf = out_bytes(rows, K, 2), out_bytes(rows, K, 32)
    nv.nvfp4_mx_quantize_rows_bf16(None, tok, 0, q, sf, rows, 0, K)
    assert (host(q) == 0).all() and (host(sf) == 0).all()


@pytest.mark.parametrize("T,E,k,first,local", [(64, 8, 4, 0, 8), (33, 16, 3, 4, 8)])
def test_routing_and_row_order_feed_the_nvfp4_experts(T, E, k, first, local):
    # logits -> nvfp4_moe_route -> nvfp4_moe_sort -> nvfp4_moe_ffn, for all experts or a range of them
    H, I = 1024, 512
    say("route, sort, NVFP4 experts", T, E, k, first, local)
    P = _ffn_problem(T, H, I, local, k, seed=500 + T)
    logits = np.random.default_rng(T).standard_normal((T, E)).astype(np.float32)
    i32 = lambda *n: torch.full(n, -7, dtype=torch.int32, device="cuda")
    ids, off, tok, rows = i32(T, k), i32(local + 1), i32(T * k), i32(T, k)
    w = torch.zeros(T, k, device="cuda")
    nv.nvfp4_moe_route(dev(logits), None, nv.SCORE_SOFTMAX, 1, 1, 1, k, True, 1.0, ids, w, T, E)
    nv.nvfp4_moe_sort(ids, first, off, tok, rows, T, local, k, nv.moe_sort_workspace(T, local, k))
    t = {n: dev(P[n]) for n in ("a_gu", "a_d")}
    pgu, pgusf = nv.grouped_pack(dev(P["w_gu"]), dev(P["w_gu_sf"]), 2 * I, H, local)
    pd, pdsf = nv.grouped_pack(dev(P["w_d"]), dev(P["w_d_sf"]), H, I, local)
    ws = torch.zeros(nv.nvfp4_moe_ffn_workspace_size(T, H, I, k), dtype=torch.uint8, device="cuda")
    out = torch.empty((T, H), dtype=torch.int16, device="cuda")
    status = torch.full((1,), -7, dtype=torch.int32, device="cuda")
    args = (dev(P["x"].view(np.int16)), scalar(P["gs_x"]), tok, off, pgu, pgusf, t["a_gu"], scalar(P["gs_h"]), pd, pdsf, t["a_d"],
            rows, w, out, T, H, I, local, k, ws, status)
    nv.nvfp4_moe_ffn(*args)
    # its status looks at every row's token, and the row order leaves those behind the last expert as they were
    valid = int(host(off)[-1])
    assert host(status)[0] == (0 if valid == T * k else -(1 + valid))
    first_out = bits(out).copy()
    tok[valid:] = 0
    out.zero_()
    nv.nvfp4_moe_ffn(*args)
    assert host(status)[0] == 0
    np.testing.assert_array_equal(bits(out), first_out)
    want_ids, want_w = x.route(logits, None, x.SOFTMAX, 1, 1, 1, k, True, 1.0)
    np.testing.assert_array_equal(host(ids), want_ids)
    want_off, want_tok, want_rows = x.sort_rows(want_ids, first, local)
    np.testing.assert_array_equal(host(off), want_off)
    np.testing.assert_array_equal(host(rows), want_rows)
    np.testing.assert_array_equal(host(tok)[:valid], want_tok)
    want_tok = np.concatenate([want_tok, np.zeros(T * k - want_tok.size, np.int32)])
    ref, _ = m.moe_ffn(P["x"], P["gs_x"], want_tok, want_off, P["w_gu"], P["w_gu_sf"], P["a_gu"], P["gs_h"], P["w_d"],
                       P["w_d_sf"], P["a_d"], want_rows, want_w.astype(np.float32), I)
    fr = _frob(bits(out), ref)
    say("relative Frobenius error", fr)
    assert fr <= 1e-2  # the bound of nvfp4_moe_ffn's own test against this oracle


@pytest.mark.parametrize("counts", [[3, 0, 5], [20, 9], [30, 41], [200, 75]])  # tiles of 16, 32, 64 and 256 rows
def test_gated_outputs_at_odd_addresses(counts):
    say("gated at odd addresses", counts)
    E, rows, I, K = len(counts), sum(counts), 160, 512
    a, a_sf = dev_mx(*mx_operand(3, rows, K, lo=115, hi=123))
    b, b_sf = dev_mx(*mx_operand(4, E, 2 * I, K, lo=117, hi=125))
    off = dev(offsets_of(counts))

    def run(q, sf):
        nv.nvfp4_mx_grouped_gated_quantize(a, a_sf, None, b, b_sf, off, None, None, nv.ACT_SILU, nv.MX_FLOOR, q, sf, rows, rows, I,
                                           K, E)
    q, sf = out_bytes(rows, I, 2), out_bytes(rows, I, 32)
    run(q, sf)
    nq, ns = q.numel(), sf.numel()
    for at in (2, 6, 10):
        room, sroom = (torch.full((n + 32,), 0x5A, dtype=torch.uint8, device="cuda") for n in (nq, ns))
        run(room[at:at + nq], sroom[at // 2:at // 2 + ns])
        np.testing.assert_array_equal(host(room)[at:at + nq], host(q).reshape(-1))
        np.testing.assert_array_equal(host(sroom)[at // 2:at // 2 + ns], host(sf).reshape(-1))
        for r, lo, n in ((host(room), at, nq), (host(sroom), at // 2, ns)):
            assert (r[:lo] == 0x5A).all() and (r[lo + n:] == 0x5A).all()


@pytest.mark.parametrize("T,E,k", [(61, 30, 4), (9000, 30, 7)])  # both forms
def test_row_order_of_ids_next_to_the_largest(T, E, k):
    # experts up to id 2^31 - 1, and ids that a subtraction of the first wraps round
    first = 2 ** 31 - E
    rng = np.random.default_rng(T)
    ids = (first + rng.integers(0, E, (T, k))).astype(np.int32)
    wild = [-2 ** 31, -2 ** 31 + 1, -2 ** 31 + E, -1, 0, first - 1]
    ids.reshape(-1)[::4] = rng.choice(wild, ids.reshape(-1)[::4].shape)
    i32 = lambda n: torch.full((n,), -7, dtype=torch.int32, device="cuda")
    off, room, rows = i32(E + 1), i32(T * k + 1), i32(T * k)
    source = i32(T * k + 1)
    source[1:] = dev(ids.reshape(-1))
    # ids and rows at odd multiples of four bytes
    nv.nvfp4_moe_sort(source[1:], first, off, room[1:], rows, T, E, k, nv.moe_sort_workspace(T, E, k))
    want = fast(ids, first, E)
    n = want[1].size
    np.testing.assert_array_equal(host(off), want[0])
    np.testing.assert_array_equal(host(rows), want[2].reshape(-1))
    np.testing.assert_array_equal(host(room)[1:n + 1], want[1])
    assert host(room)[0] == -7 and (host(room)[n + 1:] == -7).all()
