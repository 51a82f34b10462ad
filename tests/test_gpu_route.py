"""nvfp4_moe_route against the fp64 oracle: the same experts, weights within the
fp32 error of the scores."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_07_amd as nv
from oracle import experts_ref as x
from tests.gpu_util import host, say

pytestmark = pytest.mark.gpu

# relative error of a weight: a softmax score at most 35 U (two exponentials of 1 ulp with a rounded
# argument, a sum of 22 additions, a reciprocal), the same of the sum of the chosen, four more roundings
WEIGHT = 76 * 2.0 ** -24


def run(logits, bias, score, groups, top_groups, group_top, k, renorm=True, scale=1.0):
    T, E = logits.shape
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    nv.nvfp4_moe_route(logits, bias, score, groups, top_groups, group_top, k, renorm, scale, ids, w, T, E)
    return host(ids), host(w)


def check(logits, bias, score, groups, top_groups, group_top, k, renorm=True, scale=1.0):
    got, w = run(logits, bias, score, groups, top_groups, group_top, k, renorm, scale)
    want, ww = x.route(logits.float().cpu().numpy(), None if bias is None else bias.cpu().numpy(), score, groups,
                       top_groups, group_top, k, renorm, scale)
    np.testing.assert_array_equal(got, want)
    assert (np.isnan(w) == np.isnan(ww)).all()
    assert (np.abs(w - ww) <= WEIGHT * np.abs(ww) + 2.0 ** -140)[~np.isnan(ww)].all(), np.nanmax(np.abs(w / ww - 1))
    return got, w


CONFIGS = [  # T, E, groups, top_groups, group_top, k
    (1, 1, 1, 1, 1, 1), (5, 2, 1, 1, 1, 2), (3, 8, 1, 1, 1, 2), (37, 60, 1, 1, 1, 4), (9, 60, 4, 2, 2, 6),
    (64, 64, 1, 1, 1, 8), (65, 65, 5, 3, 2, 8), (130, 128, 8, 3, 1, 6), (33, 160, 8, 3, 1, 6), (257, 256, 8, 4, 2, 8),
    (7, 257, 1, 1, 1, 9), (18, 384, 1, 1, 1, 8), (6, 512, 64, 5, 2, 40), (4, 1000, 1, 1, 1, 64), (3, 1024, 32, 32, 2, 10),
    (11, 48, 48, 7, 2, 5), (11, 63, 21, 20, 2, 60),
]


@pytest.mark.parametrize("score", [nv.SCORE_SOFTMAX, nv.SCORE_SIGMOID])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,groups,top_groups,group_top,k", CONFIGS)
def test_choice_and_weights(T, E, groups, top_groups, group_top, k, with_bias, score):
    say("route", T, E, groups, top_groups, group_top, k, with_bias, score)
    g = torch.Generator(device="cuda").manual_seed(T * 1000 + E)
    logits = torch.randn(T, E, device="cuda", generator=g) * 1.5
    bias = torch.randn(E, device="cuda", generator=g) * 0.1 if with_bias else None
    check(logits, bias, score, groups, top_groups, group_top, k, True, 2.5)
    check(logits.bfloat16(), bias, score, groups, top_groups, group_top, k, False, 1.0)  # many equal logits


def test_values_that_fp32_cannot_tell_apart():
    # biases that bring every score to about 0.9: what decides is the rounding of the bias itself
    g = torch.Generator(device="cuda").manual_seed(3)
    for score, E, groups, kept, top in ((nv.SCORE_SIGMOID, 256, 8, 4, 2), (nv.SCORE_SIGMOID, 100, 1, 1, 1),
                                        (nv.SCORE_SOFTMAX, 128, 4, 2, 2), (nv.SCORE_SOFTMAX, 600, 1, 1, 1)):
        row = torch.randn(1, E, device="cuda", generator=g)
        s = torch.softmax(row.double(), -1) if score == nv.SCORE_SOFTMAX else torch.sigmoid(row.double())
        bias = (0.9 - s[0]).float()
        v = s[0] + bias.double()
        assert v.unique().numel() > E // 2 and float(v.max() - v.min()) < 2e-7
        check(row.repeat(6, 1), bias, score, groups, kept, top, 8)


def test_ties_take_the_lowest_index():
    logits = torch.zeros(3, 256, device="cuda")
    logits[1, 100:130] = 1.0
    logits[2] = torch.arange(256, device="cuda") // 16 % 2
    for groups, kept, top in ((1, 1, 1), (8, 4, 2), (16, 3, 1)):
        for bias in (None, torch.zeros(256, device="cuda"), torch.full((256,), 0.25, device="cuda")):
            for score in (nv.SCORE_SOFTMAX, nv.SCORE_SIGMOID):
                check(logits, bias, score, groups, kept, top, 8)


def test_infinities_and_nan():
    inf, nan = float("inf"), float("nan")
    logits = torch.randn(8, 40, device="cuda", generator=torch.Generator(device="cuda").manual_seed(4))
    logits[0] = -inf
    logits[1, 5:] = -inf          # fewer finite than top_k
    logits[2, 3] = nan
    logits[3, 3] = inf
    logits[4] = nan
    logits[5, ::2] = -3.0e38
    logits[7] = -inf              # no finite one, and NaN
    logits[7, 2:30:3] = nan
    bias = torch.zeros(40, device="cuda")
    bias[7], bias[8] = -inf, -3e38
    for b in (None, bias):
        for score in (nv.SCORE_SOFTMAX, nv.SCORE_SIGMOID):
            for groups, kept, top in ((1, 1, 1), (4, 2, 2), (4, 3, 1)):
                for renorm in (True, False):
                    ids, _ = run(logits, b, score, groups, kept, top, 8, renorm)
                    want, ww = x.route(logits.cpu().numpy(), None if b is None else b.cpu().numpy(), score, groups, kept,
                                       top, 8, renorm, 1.0)
                    assert all(len(set(r)) == 8 and min(r) >= 0 and max(r) < 40 for r in ids.tolist())
                    finite = [1, 5, 6] if score == nv.SCORE_SOFTMAX else list(range(8))
                    np.testing.assert_array_equal(ids[finite], want[finite], err_msg=f"{score} {groups} {b is None}")
                    np.testing.assert_array_equal(ids[0], want[0])
    w = run(logits, None, nv.SCORE_SOFTMAX, 1, 1, 1, 8)[1]
    assert (w[0] == 0).all() and np.isnan(w[2]).all() and np.isnan(w[3]).any() and np.isnan(w[4]).all()


def test_row_strides_other_stream_and_graph():
    g = torch.Generator(device="cuda").manual_seed(5)
    wide = torch.randn(50, 301, device="cuda", generator=g)
    for t in (wide[:, 3:259], wide.bfloat16()[:, 1:257], wide.bfloat16()[:, 44:300]):
        check(t, None, nv.SCORE_SOFTMAX, 8, 4, 2, 8)
    logits = wide[:, :256].contiguous()
    bias = torch.zeros(256, device="cuda")
    ids, w = torch.empty(50, 8, dtype=torch.int32, device="cuda"), torch.empty(50, 8, device="cuda")
    args = (logits, bias, nv.SCORE_SIGMOID, 8, 4, 2, 8, True, 1.0, ids, w, 50, 256)
    nv.nvfp4_moe_route(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.nvfp4_moe_route(*args)
    for _ in range(3):
        logits.copy_(torch.randn(50, 256, device="cuda", generator=g))
        graph.replay()
        torch.cuda.synchronize()
        got, gw = host(ids).copy(), host(w).copy()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        ids.zero_()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            nv.nvfp4_moe_route(*args)
        torch.cuda.current_stream().wait_stream(s)
        np.testing.assert_array_equal(got, host(ids))
        np.testing.assert_array_equal(gw, host(w))


def test_refused_tensors():
    logits = torch.randn(4, 8, device="cuda")
    ids, w = torch.empty(4, 2, dtype=torch.int32, device="cuda"), torch.empty(4, 2, device="cuda")

    def call(**kw):
        a = dict(logits=logits, bias=None, score=0, n_group=1, topk_group=1, group_top=1, top_k=2, renormalize=True, scale=1.0,
                 ids=ids, weights=w, T=4, E=8)
        a.update(kw)
        return nv.nvfp4_moe_route(**a)
    call()
    for bad in (dict(logits=logits.half()), dict(logits=logits.cpu()), dict(logits=logits.t()), dict(T=5), dict(E=9),
                dict(ids=ids.long()), dict(ids=ids[:, :1]), dict(weights=w.double()), dict(bias=torch.zeros(7, device="cuda")),
                dict(bias=torch.zeros(8, device="cuda").bfloat16()), dict(top_k=9), dict(logits=None)):
        with pytest.raises(nv.Nvfp4Error):
            call(**bad)


@pytest.mark.parametrize("score", [nv.SCORE_SOFTMAX, nv.SCORE_SIGMOID])
def test_weights_of_far_logits(score):
    # every expert is chosen, with weights down to where fp32 ends (below 2^-126 they may be 0)
    g = torch.Generator(device="cuda").manual_seed(6)
    for E in (5, 32, 64):
        logits = torch.randn(20, E, device="cuda", generator=g) * 30
        for renorm in (True, False):
            got, w = run(logits, None, score, 1, 1, 1, E, renorm)
            want, ww = x.route(logits.cpu().numpy(), None, score, 1, 1, 1, E, renorm, 1.0)
            if score == nv.SCORE_SOFTMAX:  # a sigmoid of more than 37 is 1 in 64 bits, a tie
                np.testing.assert_array_equal(got, want)
            else:
                np.testing.assert_array_equal(np.sort(got, 1), np.sort(want, 1))
                w, ww = (np.take_along_axis(a, np.argsort(i, 1), 1) for a, i in ((w, got), (ww, want)))
            # 8 U a score (an exponential within 3, a sum or 1 + it, a reciprocal, a product), the sum's 11
            # additions of at most 64 of them, its own reciprocal and product
            assert (np.abs(w - ww) <= 34 * 2.0 ** -24 * ww + 2.0 ** -125).all(), np.max(np.abs(w / ww - 1))


def test_renormalised_weights_of_scores_below_fp32():
    # the bias chooses experts whose scores are 1e-30 .. 1e-300
    for score in (nv.SCORE_SOFTMAX, nv.SCORE_SIGMOID):
        for far in (70.0, 87.0, 95.0, 103.0, 300.0, 690.0):
            logits = torch.zeros(3, 40, device="cuda")
            logits[:, 10:20] = -far - torch.arange(10, device="cuda") / 8
            logits[1, 10:20] -= 3
            logits[2, :10] = 40.0
            bias = torch.zeros(40, device="cuda")
            bias[10:20] = 2 + torch.arange(10, device="cuda") / 4
            got, w = run(logits, bias, score, 1, 1, 1, 6)
            l, b = logits.cpu().numpy(), bias.cpu().numpy()
            want, ww = x.route(l, b, score, 1, 1, 1, 6, True, 1.0)
            np.testing.assert_array_equal(got, want)
            # Softmax at 690 + 40: scores of 2^-1058, whose 64-bit steps of 2^-1074 are 2^-16 of them.  An
            # exponential and a product round to such steps, here and in the oracle, by half a step each; a
            # weight has them in its score and, averaged, in the sum: 8 halves, 4 steps of the smallest score.
            least = np.take_along_axis(x.scores(l, score), want.astype(np.int64), 1).min(1, keepdims=True)
            steps = 4 * 2.0 ** -1074 / least
            assert (np.abs(w - ww) <= (WEIGHT + steps) * ww).all(), (score, far, np.abs(w / ww - 1).max(1), steps)
    # below what 64 bits hold they are 0
    assert (run(logits - 1e30, torch.zeros(40, device="cuda"), nv.SCORE_SIGMOID, 1, 1, 1, 6)[1] == 0).all()
