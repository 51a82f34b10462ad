"""nvfp4_moe_route where fp32 ends: renormalised weights of chosen scores far
apart, group sums of values that cancel, and the last choice of as many as
there may be."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_07_amd as nv
from oracle import experts_ref as x
from tests.gpu_util import dev, host, say
from tests.test_gpu_route import WEIGHT, check, run

pytestmark = pytest.mark.gpu


def weights_near(logits, bias, score, k, scale):
    got, w = run(dev(logits), None if bias is None else dev(bias), score, 1, 1, 1, k, True, scale)
    want, ww = x.route(logits, bias, score, 1, 1, 1, k, True, scale)
    np.testing.assert_array_equal(got, want)
    # the error of a weight, and half a step of fp32 below 2^-126
    assert (np.abs(w - ww) <= WEIGHT * ww + 2.0 ** -150).all(), (score, k, scale, w, ww)


@pytest.mark.parametrize("scale", [1.0, 2.0 ** 40])
@pytest.mark.parametrize("score", [nv.SCORE_SOFTMAX, nv.SCORE_SIGMOID])
def test_renormalised_weights_of_scores_far_apart(score, scale):
    # the bias chooses experts of these logits: some of their scores are below 2^-126, their sum is not
    for chosen in ([-61.0, -95.0], [-40.0, -88.0, -89.0], [-62.0, -63.0, -130.0], [-87.0, -87.5], [-3.0, -100.0, -101.0],
                   [20.0, -95.0, -61.0]):
        say("far apart", score, scale, chosen)
        k = len(chosen)
        logits = np.zeros((2, 40), np.float32)
        logits[:, 10:10 + k] = chosen
        logits[1, 39] = 5.0
        bias = np.zeros(40, np.float32)
        bias[10:10 + k] = 8.0 - np.arange(k)
        weights_near(logits, bias, score, k, scale)


@pytest.mark.parametrize("scale", [1.0, 2.0 ** 40])
def test_renormalised_weights_without_bias(scale):
    # all experts are chosen, the sum is about 1, and weights times the scale are ordinary numbers
    logits = -np.array([[0, 1, 30, 80, 87, 88, 95, 100], [0, 90, 91, 92, 93, 94, 95, 96]], np.float32)
    for score in (nv.SCORE_SOFTMAX, nv.SCORE_SIGMOID):
        weights_near(logits, None, score, 8, scale)


def test_group_sums_that_cancel():
    # groups of two whose biases are opposite: the sums are those of the scores, the values are
    # thousands, and fp32 has steps of 2^-14 there
    rng = np.random.default_rng(7)
    for score in (nv.SCORE_SOFTMAX, nv.SCORE_SIGMOID):
        for high, groups, kept in ((1000.0, 32, 16), (50.0, 64, 9), (3.0e6, 8, 3)):
            say("cancelling", score, high, groups, kept)
            logits = (rng.standard_normal((40, 2 * groups)) * 0.5 / np.sqrt(high)).astype(np.float32)
            bias = np.zeros(2 * groups, np.float32)
            bias[0::2] = high + np.arange(groups) * max(1.0, high / 1000)
            bias[1::2] = -bias[0::2]
            check(dev(logits), dev(bias), score, groups, kept, 2, min(kept, 8))


def border(rng, score, E, k):
    """Logits and biases whose values are 0.01 apart but for the k-th and the one after it, which differ
    by less than fp32 sees: the one of the higher index is the larger."""
    for _ in range(1000):
        logits = rng.standard_normal((1, E)).astype(np.float32)
        order = rng.permutation(E)
        target = np.empty(E)
        target[order] = 0.5 + 0.01 * np.arange(E, 0, -1)
        p, q = sorted(order[k - 1:k + 1])
        target[q] = target[p] = target[order[k - 1]]
        s = x.scores(logits, score)[0]
        bias = (target - s).astype(np.float32)
        v = s + bias
        if 0 < v[q] - v[p] < 2e-8:
            return logits, bias
    raise AssertionError("no such pair")


@pytest.mark.parametrize("score", [nv.SCORE_SOFTMAX, nv.SCORE_SIGMOID])
@pytest.mark.parametrize("E,k", [(65, 64), (100, 64), (1000, 64), (100, 63), (64, 63), (40, 1), (60, 8)])
def test_last_choice_that_fp32_cannot_tell(E, k, score):
    say("border", E, k, score)
    rng = np.random.default_rng(E + k)
    for _ in range(5):
        logits, bias = border(rng, score, E, k)
        check(dev(np.repeat(logits, 3, 0)), dev(bias), score, 1, 1, 1, k)
