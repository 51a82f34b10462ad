"""Pins of the block oracle (oracle.block_ref) against torch's own fp64
operations on the CPU, and of its bounds against fp32 evaluations."""
import numpy as np
import pytest
import torch

from oracle import block_ref as br
from oracle import nvfp4_ref as o

F = torch.nn.functional


@pytest.mark.parametrize("act,f", [(br.ACT_NONE, lambda x: x), (br.ACT_RELU, F.relu), (br.ACT_GELU, F.gelu),
                                   (br.ACT_GELU_TANH, lambda x: F.gelu(x, approximate="tanh")), (br.ACT_SILU, F.silu)])
def test_activations(act, f):
    x = np.concatenate([np.linspace(-30, 30, 20001), [0.0, -0.0, 1e-30, -1e-30, 300.0, -300.0]])
    want = f(torch.from_numpy(x)).numpy()
    # torch forms 1 + erf and 1 + tanh, which cancel for negative x: absolute there
    np.testing.assert_allclose(br.activation(x, act), want, rtol=1e-13, atol=1e-14)
    x32 = x.astype(np.float32)
    y = br.activation(x32, act)
    # an fp32 evaluation lies within the bound of the activation's own steps where nothing cancels
    pos = x32 >= 0
    got = f(torch.from_numpy(x32)).numpy().astype(np.float64)
    assert (np.abs(got - y)[pos] <= br._act_error(x32.astype(np.float64), y, act, np.zeros(len(x)))[pos] + br.U * np.abs(y)[pos]).all()


def test_epilogue_and_gated_values_and_bounds():
    rng = np.random.default_rng(5)
    M, N, K = 9, 24, 512
    xa, xb = rng.standard_normal((M, K)), rng.standard_normal((2 * N, K))
    bias, res = rng.standard_normal(2 * N), rng.standard_normal((M, N))
    t = lambda v: torch.from_numpy(v)
    y, err = br.epilogue(xa, xb[:N], 0.5, bias[:N], br.ACT_GELU, res, 0.25)
    want = F.gelu(0.5 * t(xa) @ t(xb[:N]).T + t(bias[:N])) + 0.25 * t(res)
    np.testing.assert_allclose(y, want.numpy(), rtol=1e-12, atol=1e-12)
    h, herr = br.gated(xa, xb[:N], xb[N:], (0.5, 2.0), bias, br.ACT_SILU)
    lin = lambda w, a, b: a * t(xa) @ t(w).T + t(b)
    want_h = F.silu(lin(xb[:N], 0.5, bias[:N])) * lin(xb[N:], 2.0, bias[N:])
    np.testing.assert_allclose(h, want_h.numpy(), rtol=1e-12, atol=1e-12)
    # fp32 evaluations of the same steps lie within the bounds, and the bounds are below a bf16 step of the sums
    a32, b32 = xa.astype(np.float32), xb.astype(np.float32)
    x64a, x64b = a32.astype(np.float64), b32.astype(np.float64)
    bias32, res32 = bias.astype(np.float32), res.astype(np.float32)
    y, err = br.epilogue(x64a, x64b[:N], 0.5, bias32[:N].astype(np.float64), br.ACT_SILU, res32.astype(np.float64), 0.25)
    s = np.float32(0.5) * (a32 @ b32[:N].T) + bias32[:N]
    got = s / (1 + np.exp(-s)) + np.float32(0.25) * res32
    assert (np.abs(got - y) <= err).all()
    assert err.max() < 2.0 ** -8 * np.abs(y).max()


@pytest.mark.parametrize("kind", [br.RMS, br.LAYER])
def test_norms(kind):
    rng = np.random.default_rng(6)
    T, H = 11, 272
    bf = lambda v: torch.from_numpy(v.astype(np.float32)).to(torch.bfloat16).float().numpy()
    x, res = bf(rng.standard_normal((T, H)) * 2 + 1), bf(rng.standard_normal((T, H)))
    pw, w = bf(1 + 0.2 * rng.standard_normal(H)), bf(1 + 0.2 * rng.standard_normal(H))
    pb, b = (bf(rng.standard_normal(H)), bf(rng.standard_normal(H))) if kind == br.LAYER else (None, None)
    gate = bf(rng.standard_normal((3, H)))
    args = (x, pw, pb, gate, 4, res, 0.5, w, b, 1e-5, kind)
    t = lambda v: None if v is None else torch.from_numpy(v).double()

    def norm(v, w_, b_):
        if kind == br.LAYER:
            return F.layer_norm(v, (H,), t(w_), t(b_), 1e-5)
        return F.rms_norm(v, (H,), t(w_), 1e-5)

    r = 0.5 * t(res) + t(gate).repeat_interleave(4, 0)[:T] * norm(t(x), pw, pb)
    re, ye = br.residual_norm_exact(*args)
    np.testing.assert_allclose(re, r.numpy(), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(ye, norm(r, w, b).numpy(), rtol=1e-12, atol=1e-12)
    # the step-by-step fp32 form: at most 6 roundings to r, 5 more to y
    r32, y32 = br.residual_norm(*args)
    assert r32.dtype == y32.dtype == np.float32
    assert np.abs(r32 - re).max() <= 8 * br.U * (np.abs(re).max() + np.abs(res).max())
    assert np.abs(y32 - ye).max() <= 64 * br.U * (np.abs(ye).max() + 1)


def test_quantized_range_and_check():
    rng = np.random.default_rng(7)
    h = rng.standard_normal((40, 64)).astype(np.float32).astype(np.float64)
    gs = np.float32(2688.0 / np.abs(h).max())
    q, sf = o.quantize(h.astype(np.float32), gs)
    err = np.full_like(h, 1e-6)
    br.check_quantized(q, sf, h, err, gs)
    # a code one step off, and a scale one step off, are found
    bad = q.copy()
    bad[3, 5] = (bad[3, 5] & 0xF0) | ((bad[3, 5] + 2) & 0x7)
    with pytest.raises(AssertionError):
        br.check_quantized(bad, sf, h, err, gs)
    bad = sf.copy()
    bad[4, 1] += 1
    with pytest.raises(AssertionError):
        br.check_quantized(q, bad, h, err, gs)
