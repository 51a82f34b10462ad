"""A mixture-of-experts layer as it is used: routing, row order and the experts'
feed-forward in a row."""
import threading

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_07_amd as nv
from oracle import experts_ref as x
from tests.experts_util import dev_mx, mx_operand
from tests.gpu_util import dev, host, say

pytestmark = pytest.mark.gpu


class Layer:
    def __init__(self, seed, T, H, I, E, k, groups=1, kept=1, extras=False, first=0, local=None):
        rng = np.random.default_rng(seed)
        self.T, self.H, self.I, self.E, self.k, self.groups, self.kept = T, H, I, E, k, groups, kept
        self.first, self.local = first, E if local is None else local
        L = self.local
        self.np = dict(
            logits=rng.standard_normal((T, E)).astype(np.float32), bias=(rng.standard_normal(E) * 0.05).astype(np.float32),
            x=torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).bfloat16().float().numpy())
        self.np["gu"], self.np["gu_sf"] = mx_operand(seed + 1, L, 2 * I, H, lo=119, hi=121)
        self.np["dn"], self.np["dn_sf"] = mx_operand(seed + 2, L, H, I, lo=119, hi=121)
        self.extras = extras
        f32 = lambda *s: rng.uniform(0.5, 1.5, s).astype(np.float32)
        bf = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).bfloat16().float().numpy()
        if extras:
            self.np.update(al=f32(2 * L), ald=f32(L), bg=bf(L, 2 * I), bd=bf(L, H))
        self.t = {n: dev(v) for n, v in self.np.items()}
        for n in ("x", "bg", "bd"):
            if n in self.t:
                self.t[n] = self.t[n].bfloat16()
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
        self.ids, self.off, self.tok, self.rows = i32(T, k), i32(L + 1), i32(T * k), i32(T, k)
        self.w = torch.zeros(T, k, device="cuda")
        self.out = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
        self.status = i32(1)
        self.sort_ws = nv.moe_sort_workspace(T, L, k)
        self.ws = nv.mx_moe_ffn_workspace(T, H, I, k)
        if self.ws is not None:
            self.ws.fill_(0xFF)

    def run(self, status=True):
        t, T, H, I, E, k = self.t, self.T, self.H, self.I, self.E, self.k
        nv.nvfp4_moe_route(t["logits"], t["bias"], nv.SCORE_SIGMOID, self.groups, self.kept, 2, k, True, 1.5, self.ids, self.w, T, E)
        nv.nvfp4_moe_sort(self.ids, self.first, self.off, self.tok, self.rows, T, self.local, k, self.sort_ws)
        return nv.nvfp4_mx_moe_ffn(t["x"], self.tok, self.off, t["gu"], t["gu_sf"], t.get("al"), t.get("bg"), nv.ACT_SILU,
                                   nv.MX_FLOOR, t["dn"], t["dn_sf"], t.get("ald"), t.get("bd"), self.rows, self.w, self.out, T, H,
                                   I, self.local, k, self.ws, self.status if status else None)

    def want(self):
        n = self.np
        ids, w = x.route(n["logits"], n["bias"], x.SIGMOID, self.groups, self.kept, 2, self.k, True, 1.5)
        off, tok, rows = x.sort_rows(ids, self.first, self.local)
        tok = np.concatenate([tok, np.zeros(self.T * self.k - tok.size, np.int32)])
        return x.moe_ffn(n["x"], tok, off, n["gu"], n["gu_sf"], n.get("al"), n.get("bg"), 4, x.FLOOR, n["dn"], n["dn_sf"],
                         n.get("ald"), n.get("bd"), rows, w)


def near(got, want):
    g = got.double().cpu().numpy()
    assert np.isfinite(g).all()
    return np.linalg.norm(g - want) / np.linalg.norm(want)


@pytest.mark.parametrize("T,H,I,E,k,groups,kept,extras", [
    (1, 256, 256, 8, 2, 1, 1, False), (5, 512, 256, 16, 4, 4, 2, True), (33, 768, 512, 12, 3, 1, 1, True),
    (64, 256, 768, 4, 2, 2, 2, False), (300, 512, 256, 3, 2, 1, 1, True)])
def test_layer_against_the_oracle(T, H, I, E, k, groups, kept, extras):
    say("layer", T, H, I, E, k)
    l = Layer(T + E, T, H, I, E, k, groups, kept, extras)
    out = l.run()
    # the output's rounding (2^-8 = 3.9e-3 at most), and hidden codes that fall to the other side of a border
    assert near(out, l.want()) <= 5e-3
    assert host(l.status)[0] == 0
    # the same steps called one by one give the same bits
    first = host(out.view(torch.int16)).copy()
    rows = T * k
    u8 = lambda r, c: torch.empty(r, c, dtype=torch.uint8, device="cuda")
    xq, xsf, hq, hsf = u8(T, H // 2), u8(T, H // 32), u8(rows, I // 2), u8(rows, I // 32)
    down, again = torch.empty(rows, H, dtype=torch.bfloat16, device="cuda"), torch.empty_like(out)
    t = l.t
    nv.nvfp4_mx_quantize_rows_bf16(t["x"], None, nv.MX_FLOOR, xq, xsf, T, T, H)
    nv.nvfp4_mx_grouped_gated_quantize(xq, xsf, l.tok, t["gu"], t["gu_sf"], l.off, t.get("al"), t.get("bg"), nv.ACT_SILU,
                                       nv.MX_FLOOR, hq, hsf, rows, T, I, H, E)
    nv.nvfp4_mx_grouped_gemm(hq, hsf, None, t["dn"], t["dn_sf"], l.off, t.get("ald"), t.get("bd"), down, rows, rows, H, I, E)
    nv.nvfp4_moe_combine(down, l.rows, l.w, again, T, H, k, rows)
    np.testing.assert_array_equal(host(again.view(torch.int16)), first)
    # and again
    l.out.zero_()
    np.testing.assert_array_equal(host(l.run().view(torch.int16)), first)


def test_experts_of_two_gpus_add_up():
    # each holds half of the experts: its rows only, the others' weights add nothing
    a, b, full = (Layer(70, 40, 512, 256, 16, 4, 4, 2, False, f, n) for f, n in ((0, 8), (8, 8), (0, 16)))
    for l, lo in ((a, 0), (b, 8)):
        for n in ("gu", "gu_sf", "dn", "dn_sf"):
            l.np[n] = full.np[n][lo:lo + 8]
            l.t[n] = dev(l.np[n])
    got = [l.run().double().cpu().numpy() for l in (a, b)]
    assert host(a.off)[-1] + host(b.off)[-1] == 160 and (host(a.rows) < 0).any() and (host(b.rows) < 0).any()
    want = full.want()
    assert np.linalg.norm(got[0] + got[1] - want) / np.linalg.norm(want) <= 5e-3
    assert near(a.out, a.want()) <= 5e-3


@pytest.mark.parametrize("T,E,k", [(17, 32, 4), (333, 8, 4), (1000, 4, 2)])
def test_captured_and_replayed(T, E, k):
    l = Layer(80, T, 512, 512, E, k, 4, 2, True)
    l.run(False)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        l.run(False)
    g = torch.Generator(device="cuda").manual_seed(1)
    for _ in range(4):
        l.t["logits"].copy_(torch.randn(T, E, device="cuda", generator=g))
        l.t["x"].copy_(torch.randn(T, 512, device="cuda", generator=g))
        l.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = host(l.out.view(torch.int16)).copy()
        l.out.zero_()
        l.run()
        np.testing.assert_array_equal(host(l.out.view(torch.int16)), got)


@pytest.mark.timeout(120)
def test_threads_on_streams_of_their_own():
    layers = [Layer(90, 1, 512, 256, 16, 4), Layer(91, 100, 256, 512, 8, 2), Layer(92, 33, 768, 256, 5, 3)]
    want = [l.run().clone() for l in layers]
    torch.cuda.synchronize()
    wrong, errors = [], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    layers[i].out.zero_()
                    layers[i].run()
                    torch.cuda.current_stream().synchronize()
                    if not torch.equal(layers[i].out, want[i]):
                        wrong.append(i)
                        return
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and not wrong


def test_no_routed_rows():
    l = Layer(93, 6, 256, 256, 4, 2)
    l.run()
    # ids that no expert here has: every row left out, zeros come out
    l.ids.fill_(-1)
    nv.nvfp4_moe_sort(l.ids, 0, l.off, l.tok, l.rows, 6, 4, 2, l.sort_ws)
    l.out.fill_(7.0)
    t = l.t
    args = (t["gu"], t["gu_sf"], None, None, 4, 0, t["dn"], t["dn_sf"], None, None)
    nv.nvfp4_mx_moe_ffn(t["x"], l.tok, l.off, *args, l.rows, l.w, l.out, 6, 256, 256, 4, 2, l.ws, l.status)
    assert (host(l.out.float()) == 0).all() and host(l.status)[0] == 0
    l.out.fill_(7.0)
    nv.nvfp4_mx_moe_ffn(t["x"], None, l.off, *args, None, None, l.out, 6, 256, 256, 4, 0, l.ws)
    assert (host(l.out.float()) == 0).all()


def test_refused_tensors():
    l = Layer(94, 6, 256, 256, 4, 2)
    l.run()
    t = l.t

    def call(**kw):
        a = dict(x=t["x"], row_token=l.tok, offsets=l.off, w_gu=t["gu"], w_gu_sf=t["gu_sf"], alpha_gu=None, bias_gu=None, act=4,
                 rule=0, w_d=t["dn"], w_d_sf=t["dn_sf"], alpha_d=None, bias_d=None, token_rows=l.rows, token_weight=l.w, out=l.out,
                 T=6, H=256, I=256, E=4, top_k=2, workspace=l.ws)
        a.update(kw)
        return nv.nvfp4_mx_moe_ffn(**a)
    call()
    for bad in (dict(x=t["x"].float()), dict(row_token=l.tok[:11]), dict(offsets=l.off[:4]), dict(w_gu=t["gu"][:3]),
                dict(w_gu_sf=t["gu_sf"][:3]), dict(w_d=t["dn"][:3]), dict(w_d_sf=t["dn_sf"][:3]), dict(token_rows=l.rows[:5]),
                dict(token_weight=l.w[:5]), dict(token_weight=l.w.double()), dict(out=l.out[:5]), dict(workspace=l.ws[:256]),
                dict(workspace=None), dict(T=7), dict(top_k=3), dict(E=5), dict(alpha_gu=torch.ones(4, device="cuda")),
                dict(bias_d=torch.ones(4, 256, device="cuda")), dict(token_rows=l.rows.long())):
        with pytest.raises(nv.Nvfp4Error):
            call(**bad)
