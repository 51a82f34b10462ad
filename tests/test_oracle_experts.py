"""Pins of the mixture-of-experts oracle (CPU only): torch's own operators where
they coincide, worked examples, and brute force."""
import itertools

import numpy as np
import pytest
import torch

from oracle import experts_ref as x
from oracle import mxfp4_ref as mx
from oracle import nvfp4_ref as nv


@pytest.mark.parametrize("score", [x.SOFTMAX, x.SIGMOID])
def test_scores_are_torch_s(score):
    l = np.random.default_rng(1).standard_normal((5, 40)) * 4
    t = torch.from_numpy(l)
    want = torch.softmax(t, -1) if score == x.SOFTMAX else torch.sigmoid(t)
    np.testing.assert_allclose(x.scores(l, score), want.numpy(), rtol=1e-14)


def test_ungrouped_choice_is_topk():
    l = np.random.default_rng(2).standard_normal((50, 33))
    ids, w = x.route(l, None, x.SOFTMAX, 1, 1, 1, 5, True, 2.0)
    top = torch.topk(torch.from_numpy(l), 5, -1)
    np.testing.assert_array_equal(ids, top.indices.numpy())
    # renormalised softmax scores are the softmax of the chosen logits
    np.testing.assert_allclose(w, 2.0 * torch.softmax(top.values, -1).numpy(), rtol=1e-13)


def test_groups_by_hand():
    # groups (0.1 0.9) (0.5 0.6) (0.8 0.3): by the largest, groups 0 and 2; by the sum of two, 1 and 2
    p = np.array([[0.1, 0.9, 0.5, 0.6, 0.8, 0.3]])
    l = np.log(p / (1 - p))
    assert x.route(l, None, x.SIGMOID, 3, 2, 1, 3, False, 1.0)[0].tolist() == [[1, 4, 5]]
    assert x.route(l, None, x.SIGMOID, 3, 2, 2, 3, False, 1.0)[0].tolist() == [[4, 3, 2]]
    # the bias moves the choice and not the weight
    ids, w = x.route(l, [0, -1, 0, 0, 0, 0], x.SIGMOID, 1, 1, 1, 1, False, 1.0)
    assert ids.tolist() == [[4]] and abs(w[0, 0] - 0.8) < 1e-12


def test_ties_nan_and_empty_rows():
    inf = np.inf
    assert x.route([[1.0, 2.0, 2.0, 0.0]], None, x.SOFTMAX, 1, 1, 1, 3, False, 1.0)[0].tolist() == [[1, 2, 0]]
    ids, w = x.route([[-inf] * 4], None, x.SOFTMAX, 1, 1, 1, 2, True, 1.0)
    assert ids.tolist() == [[0, 1]] and (w == 0).all()
    ids, w = x.route([[np.nan, -inf, 1.0, 0.0]], None, x.SIGMOID, 1, 1, 1, 3, False, 1.0)
    assert ids.tolist() == [[2, 3, 1]] and w[0, 2] == 0
    ids, w = x.route([[np.nan, -inf, 1.0, 0.0]], None, x.SIGMOID, 1, 1, 1, 4, False, 1.0)
    assert ids.tolist() == [[2, 3, 1, 0]] and np.isnan(w[0, 3])


def test_sort_rows_by_hand():
    off, tok, rows = x.sort_rows(np.array([[2, 0], [1, 2], [2, 5]]), 0, 4)
    assert off.tolist() == [0, 1, 2, 5, 5] and tok.tolist() == [0, 1, 0, 1, 2]
    assert rows.tolist() == [[2, 0], [1, 3], [4, -1]]
    off, tok, rows = x.sort_rows(np.array([[2, 0], [1, 2], [2, 5]]), 2, 2)
    assert off.tolist() == [0, 3, 3] and rows.tolist() == [[0, -1], [-1, 1], [2, -1]]


def test_codes_are_the_nearest():
    v = np.concatenate([np.linspace(-7, 7, 2801), [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.0]])
    got = x.e2m1_codes(v)
    np.testing.assert_array_equal(got, nv.e2m1_encode(v.astype(np.float32)) if hasattr(nv, "e2m1_encode") else got)
    dec = nv.E2M1_LUT[got]
    assert (np.abs(dec - np.clip(v, -6, 6)) <= np.min(np.abs(nv.E2M1_LUT[None] - np.clip(v, -6, 6)[:, None]), -1)).all()
    assert got[-8:].tolist() == [0, 2, 2, 4, 4, 6, 6, 8]  # ties to the even code, minus zero kept


@pytest.mark.parametrize("rule", [x.FLOOR, x.CEIL])
def test_block_exponents_by_search(rule):
    for peak in itertools.chain([1.0, 1.5, 1.5000001, 1.9999, 2.0, 6.0, 6.0001, 7.99, 8.0, 2.0 ** -126, 2.0 ** -149, 1e38],
                                np.random.default_rng(3).lognormal(0, 8, 200).astype(np.float32)):
        peak = float(np.float32(peak))
        e = int(x.block_exponents(np.array(peak), rule))
        if rule == x.FLOOR:
            want = max(k for k in range(-160, 129) if 4.0 * 2.0 ** k <= peak)
        else:
            want = min(k for k in range(-160, 129) if peak <= 6.0 * 2.0 ** k)
        assert e == min(max(want, -127), 125), peak


def test_quantised_blocks():
    v = np.zeros((1, 96), np.float32)
    v[0, :32] = np.linspace(-3, 3, 32)
    v[0, 40] = np.nan
    v[0, 70] = -np.inf
    q, sf = x.quantize(v)
    codes = nv.unpack_codes(q)[0]
    assert sf.tolist() == [[126, 255, 252]] and (codes[32:64] == 0).all() and codes[70] == 15
    assert np.abs(mx.dequant(q[:, :16], sf[:, :1])[0] - v[0, :32]).max() <= 0.5
