"""The block operators as a layer runs them: norm -> projection -> norm with
gate and residual -> feed-forward with the residual in place -> norm, each
stage against the oracle on the stage's own inputs, eagerly and captured."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_07_amd as nv
from oracle import block_ref as br
from oracle import nvfp4_ref as o
from tests.block_util import bf16, close, dev_bf16, operand, values
from tests.gpu_util import bits, dev, host, say, scalar

pytestmark = pytest.mark.gpu

EPS = 1e-6


class Layer:
    def __init__(self, T, H, I, group, kind):
        rng = np.random.default_rng(T + H + I)
        vec = lambda m, s: bf16(rng.standard_normal(H) * s + m)
        self.T, self.H, self.I, self.group, self.kind = T, H, I, group, kind
        self.x0 = bf16(rng.standard_normal((T, H)) * 2)
        self.w = [vec(1, 0.2) for _ in range(4)]
        self.gate = bf16(rng.standard_normal((-(-T // group), H)) * 0.3 + 0.7)
        self.proj, self.gu, self.dn = operand(1, H, H), operand(3, 2 * I, H), operand(5, H, I)
        self.bias = bf16(rng.standard_normal(H))
        self.gs = np.float32(2688.0 / 8.0)  # norm outputs of a few units
        self.gs_h = np.float32(16.0)
        self.alpha = np.float32(0.01 / self.gs)
        self.alpha_gu = np.array([self.alpha, self.alpha], np.float32)
        self.alpha_d = np.float32(0.01 / self.gs_h)
        H2, H16 = H // 2, H // 16
        u8 = lambda n: torch.zeros((T, n), dtype=torch.uint8, device="cuda")
        b16 = lambda: torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
        self.d = dict(x0=dev_bf16(self.x0), w=[dev_bf16(v) for v in self.w], gate=dev_bf16(self.gate), bias=dev_bf16(self.bias),
                      proj=(dev(self.proj[0]), dev(self.proj[1])), gu=(dev(self.gu[0]), dev(self.gu[1])),
                      dn=(dev(self.dn[0]), dev(self.dn[1])), gs=scalar(self.gs), gs_h=scalar(self.gs_h),
                      alpha=scalar(self.alpha), alpha_gu=dev(self.alpha_gu), alpha_d=scalar(self.alpha_d))
        self.out = dict(q0=u8(H2), s0=u8(H16), p=b16(), x1=b16(), q1=u8(H2), s1=u8(H16), x2=b16(), y=b16())
        self.ws = nv.ffn_workspace(T, H, I)
        self.ws_p = nv.gemm_epilogue_workspace(T, H, H)

    def run(self, stages=None):
        T, H, I, d, w, t = self.T, self.H, self.I, self.d, self.d["w"], self.out
        nv.nvfp4_residual_norm(d["x0"], None, None, None, 0, None, 1.0, w[0], None, EPS, self.kind, None, None, d["gs"],
                               t["q0"], t["s0"], T, H)
        nv.nvfp4_gemm_epilogue(t["q0"], t["s0"], *d["proj"], d["alpha"], d["bias"], nv.ACT_NONE, None, 0.0, t["p"], T, H, H,
                               self.ws_p)
        nv.nvfp4_residual_norm(t["p"], w[1], None, d["gate"], self.group, d["x0"], 1.0, w[2], None, EPS, self.kind, t["x1"],
                               None, d["gs"], t["q1"], t["s1"], T, H)
        if stages is not None:
            torch.cuda.synchronize()
            stages.append({k: v.clone() for k, v in t.items()})
        # the feed-forward adds to the residual in place
        nv.nvfp4_ffn(t["q1"], t["s1"], *d["gu"], d["alpha_gu"], None, nv.ACT_SILU, d["gs_h"], *d["dn"], d["alpha_d"], None,
                     t["x1"], 1.0, t["x1"], T, H, I, self.ws)
        nv.nvfp4_residual_norm(t["x1"], None, None, None, 0, None, 1.0, w[3], None, EPS, self.kind, t["x2"], t["y"], None,
                               None, None, T, H)
        return t


CASES = [(1, 512, 768, 1, 0), (16, 6144, 2048, 4, 0), (37, 512, 256, 10, 1), (300, 768, 1024, 100, 1), (1100, 512, 4096, 1, 0)]


@pytest.mark.parametrize("T,H,I,group,kind", CASES)
def test_layer_stage_by_stage(T, H, I, group, kind):
    c = Layer(T, H, I, group, kind)
    say("layer", T, H, I, nv.nvfp4_gemm_epilogue_plan(T, H, H), nv.nvfp4_gemm_gated_plan(T, I, H), nv.nvfp4_gemm_epilogue_plan(T, H, I))
    seen = []
    end = c.run(seen)
    mid = seen[0]
    f32 = lambda t: values(t).astype(np.float32)
    # first norm, to NVFP4
    _, y = br.residual_norm(c.x0, None, None, None, 0, None, 1.0, c.w[0], None, EPS, kind)
    q, s = o.quantize(y, c.gs)
    np.testing.assert_array_equal(host(mid["q0"]), q)
    np.testing.assert_array_equal(host(mid["s0"]), s)
    # projection
    p, err = br.epilogue(o.dequant(q, s), c.proj[2], c.alpha, c.bias, 0, None, 0.0)
    close(values(mid["p"]), p, br.bf16_bound(p, err), "projection")
    # norm after it, gate, residual, norm before the feed-forward
    r, y = br.residual_norm(f32(mid["p"]), c.w[1], None, c.gate, group, c.x0, 1.0, c.w[2], None, EPS, kind)
    np.testing.assert_array_equal(bits(mid["x1"].view(torch.int16)), o.bf16_rne(r.astype(np.float64)))
    q, s = o.quantize(y, c.gs)
    np.testing.assert_array_equal(host(mid["q1"]), q)
    np.testing.assert_array_equal(host(mid["s1"]), s)
    # feed-forward: its hidden layer is rounded to 4 bits, so one step of a code near a boundary may differ
    xa = o.dequant(q, s)
    h, _ = br.gated(xa, c.gu[2][:I], c.gu[2][I:], c.alpha_gu, None, nv.ACT_SILU)
    hq, hs = o.quantize(h.astype(np.float32), c.gs_h)
    down, _ = br.epilogue(o.dequant(hq, hs), c.dn[2], c.alpha_d, None, 0, None, 0.0)
    add = values(end["x1"]) - values(mid["x1"])
    want = down + values(mid["x1"])
    # each of the two is within half a bf16 step of its own value
    step = 2.0 ** -8 * np.linalg.norm(want)
    assert np.linalg.norm(add - down) <= 1e-2 * np.linalg.norm(down) + step
    assert np.linalg.norm(down) > 4 * step, "the feed-forward's share is seen"
    # last norm: its copy of the rows and y
    x2, y = br.residual_norm(f32(end["x1"]), None, None, None, 0, None, 1.0, c.w[3], None, EPS, kind)
    np.testing.assert_array_equal(bits(end["x2"].view(torch.int16)), o.bf16_rne(x2.astype(np.float64)))
    np.testing.assert_array_equal(bits(end["y"].view(torch.int16)), o.bf16_rne(y.astype(np.float64)))


@pytest.mark.parametrize("T,H,I,group,kind", CASES[:4])
def test_layer_captured_and_on_another_stream(T, H, I, group, kind):
    c = Layer(T, H, I, group, kind)
    want = {k: v.clone() for k, v in c.run().items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for v in c.out.values():
            v.zero_()
        c.run()
    side.synchronize()
    assert all(torch.equal(want[k], c.out[k]) for k in want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run()
    for i in range(3):
        for v in c.out.values():
            v.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(want[k], c.out[k]) for k in want), f"replay {i}"
        c.run()  # the program's own eager work in between, on the same workspace
        torch.cuda.synchronize()
