"""The operators of a dense transformer block around the NVFP4 GEMM, as measured work.

Four kinds of case:

* ``epilogue``: a projection with its bias, activation and residual,
  ``d = act(alpha * A B^T + bias) + beta * residual``;
* ``gated``: both projections of a gated feed-forward block and their product,
  ``h = act(alpha[0] * A G^T + bias_g) * (alpha[1] * A U^T + bias_u)``, with the
  rows of ``b`` holding G then U;
* ``norm``: the norms around a block with its gate and residual,
  ``r = beta * residual + gate * post_norm(x)``, ``y = norm(r)``;
* ``block``: the feed-forward half of a layer as a serving loop runs it:
  residual add and norm quantised to NVFP4, then the gated feed-forward with
  an NVFP4 hidden layer, its down projection and the residual.

A and the weights are NVFP4 (two e2m1 codes per byte, one e4m3 scale per 16
elements), everything else bf16 with fp32 scalars.  ``own`` chooses between
the plain torch form (fp32, statistics in fp64) and the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
CODES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
WORKSPACE = 16 << 20      # holds the split-K exchange of any shape
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
RMS, LAYER = 0, 1


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token's attention output (or down) projection onto the residual stream
        dict(name="proj_residual_m1", op="epilogue", M=1, N=6144, K=2048, act="none", bias=False, residual=True),
        # a small batch through a biased GELU layer of a narrow model, odd sizes
        dict(name="proj_gelu_ragged", op="epilogue", M=61, N=777, K=1280, act="gelu", bias=True, residual=False),
        # a chunk of a prompt through a biased projection
        dict(name="proj_bias_residual_m1024", op="epilogue", M=1024, N=2048, K=6144, act="none", bias=True, residual=True),
        # a long prompt's square projection
        dict(name="proj_residual_m8192", op="epilogue", M=8192, N=6144, K=6144, act="none", bias=False, residual=True),
        # one token's gate and up projections
        dict(name="gated_m1", op="gated", M=1, I=2048, K=6144, act="silu", bias=False),
        # odd batch and width, biased tanh-GELU gate
        dict(name="gated_ragged", op="gated", M=333, I=1001, K=1536, act="gelu_tanh", bias=True),
        # a long prompt's gate and up projections
        dict(name="gated_m8192", op="gated", M=8192, I=8192, K=6144, act="silu", bias=False),
        # a decode batch of 16 through the feed-forward half of a layer
        dict(name="block_m16", op="block", M=16, H=6144, I=2048),
        # a prompt chunk through a wide feed-forward half
        dict(name="block_m2048", op="block", M=2048, H=6144, I=16384),
        # one token: residual add and RMS norm
        dict(name="norm_t1", op="norm", T=1, H=6144, kind=RMS, post=False, gate=0),
        # odd rows and width: layer norms on both sides, a gate for each sequence of 37 rows
        dict(name="norm_ragged", op="norm", T=777, H=1545, kind=LAYER, post=True, gate=37),
        # a long prompt: RMS norms on both sides, one gate for all rows
        dict(name="norm_t16384", op="norm", T=16384, H=6144, kind=RMS, post=True, gate=-1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["epilogue", "gated", "block", "norm"])
    if op == "norm":
        H = _log(rng, 64, 12288)
        T = _log(rng, 1, max(1, min(16384, 16384 * 6144 // H)))
        return dict(op=op, T=T, H=H, kind=rng.choice([RMS, LAYER]), post=rng.random() < 0.5,
                    gate=rng.choice([0, -1, 1, 17]))
    K = 256 * _log(rng, 1, 32)
    M = _log(rng, 1, 8192)
    if op == "block":
        return dict(op=op, M=min(M, 2048), H=K, I=256 * _log(rng, 1, 48))
    if op == "gated":
        return dict(op=op, M=M, I=_log(rng, 16, 6144), K=K, act=rng.choice(["silu", "gelu", "gelu_tanh", "relu"]),
                    bias=rng.random() < 0.5)
    return dict(op=op, M=M, N=_log(rng, 16, 6144), K=K, act=rng.choice(sorted(ACTS)), bias=rng.random() < 0.5,
                residual=rng.random() < 0.5)


def _nv(rows, k):
    return rows * k * 9 / 16  # codes and scales


def work(c):
    if c["op"] == "epilogue":
        M, N, K = c["M"], c["N"], c["K"]
        return dict(bytes=_nv(M + N, K) + 2 * M * N * (1 + c["residual"]) + 2 * N * c["bias"], flops=2 * M * N * K)
    if c["op"] == "gated":
        M, I, K = c["M"], c["I"], c["K"]
        return dict(bytes=_nv(M + 2 * I, K) + 2 * M * I + 4 * I * c["bias"], flops=4 * M * I * K)
    if c["op"] == "block":
        M, H, I = c["M"], c["H"], c["I"]
        # x, residual in; r, out; the weights (the NVFP4 activations between the calls can stay on chip)
        return dict(bytes=_nv(3 * I, H) + 2 * M * H * 4 + 2 * H, flops=6 * M * H * I)
    T, H = c["T"], c["H"]
    rows = {0: 0, -1: 1}.get(c["gate"]) if c["gate"] <= 0 else -(-T // c["gate"])
    vectors = (1 + c["post"]) * (1 + (c["kind"] == LAYER))
    return dict(bytes=2 * T * H * 4 + 2 * H * (vectors + rows), flops=8 * T * H)


# --------------------------------------------------------------- the inputs

def _quantize(x, gs):
    """fp32 [rows][K] -> e2m1 magnitudes with sign, fp32 [rows][K], and e4m3 scales [rows][K/16]:
    t = (amax / 6) * gs; sf = e4m3(t); r = gs / sf; value = e2m1(x * r)."""
    rows, K = x.shape
    b = x.reshape(rows, K // 16, 16)
    t = (b.abs().amax(-1) / 6.0 * gs).clamp(max=448.0)
    sf = t.to(torch.float8_e4m3fn)
    s = sf.float()
    r = torch.where(s == 0, torch.zeros_like(s), gs / s)
    v = b * r[..., None]
    a = v.abs().clamp(max=6.0)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    q = torch.round(a / step) * step  # ties go to the even code
    return torch.copysign(q, v).reshape(rows, K), sf


def _pack(q):
    """e2m1 values [rows][K] -> codes, uint8 [rows][K/2], element 2j in the low nibble."""
    grid = torch.tensor(CODES, device=q.device)
    code = torch.searchsorted(grid, q.abs().contiguous()) | (torch.signbit(q).long() << 3)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).to(torch.uint8).contiguous()


def _nvfp4(x):
    """Codes, scale bytes and encode scale (2688 / amax) of an fp32 matrix, by slabs of rows."""
    gs = 2688.0 / x.abs().amax()
    parts = [_quantize(s, gs) for s in x.split(4096)]
    codes = torch.cat([_pack(q) for q, _ in parts])
    return codes, torch.cat([sf.view(torch.uint8) for _, sf in parts]), gs


def _weights(g, rows, K):
    return _nvfp4(torch.randn(rows, K, device=DEV, generator=g) * 0.02)


def _bf16(g, *shape, std=1.0, mean=0.0):
    return (torch.randn(*shape, device=DEV, generator=g) * std + mean).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "norm":
        T, H = case["T"], case["H"]
        layer = case["kind"] == LAYER
        s["x"] = _bf16(g, T, H, std=2.0, mean=0.1)
        s["res"] = _bf16(g, T, H, std=3.0)
        s["w"] = _bf16(g, H, std=0.2, mean=1.0)
        s["b"] = _bf16(g, H, std=0.1) if layer else None
        s["pw"] = _bf16(g, H, std=0.2, mean=1.0) if case["post"] else None
        s["pb"] = _bf16(g, H, std=0.1) if case["post"] and layer else None
        rows = 0 if case["gate"] == 0 else 1 if case["gate"] < 0 else -(-T // case["gate"])
        s["g"] = _bf16(g, rows, H, std=0.3, mean=0.7) if rows else None
        s["r"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
        s["y"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
        return s
    if op == "block":
        M, H, I = case["M"], case["H"], case["I"]
        s["x"], s["res"] = _bf16(g, M, H, std=0.5), _bf16(g, M, H, std=2.0)
        s["w"] = _bf16(g, H, std=0.1, mean=1.0)
        s["gu"], s["gu_sf"], gu_gs = _weights(g, 2 * I, H)
        s["dn"], s["dn_sf"], dn_gs = _weights(g, H, I)
        # static activation scales, as a calibration run leaves them
        s["gs_x"] = torch.full((1,), 2688.0 / 6.0, device=DEV)
        spread = 0.02 * math.sqrt(H)
        s["gs_h"] = torch.full((1,), 2688.0 / (1.0 + 12.0 * spread * spread), device=DEV)
        s["alpha_gu"] = (1.0 / (s["gs_x"] * gu_gs)).expand(2).contiguous()
        s["alpha_dn"] = 1.0 / (s["gs_h"] * dn_gs)
        s["q"] = torch.empty(M, H // 2, dtype=torch.uint8, device=DEV)
        s["sf"] = torch.empty(M, H // 16, dtype=torch.uint8, device=DEV)
        s["r"] = torch.empty(M, H, dtype=torch.bfloat16, device=DEV)
        s["d"] = torch.empty(M, H, dtype=torch.bfloat16, device=DEV)
        s["ws"] = torch.zeros(WORKSPACE + M * I * 9 // 16 + 4096, dtype=torch.uint8, device=DEV)
        return s
    M, K = case["M"], case["K"]
    N = case["N"] if op == "epilogue" else 2 * case["I"]
    cols = N if op == "epilogue" else case["I"]
    s["a"], s["a_sf"], a_gs = _nvfp4(torch.randn(M, K, device=DEV, generator=g))
    s["w"], s["w_sf"], w_gs = _weights(g, N, K)
    s["alpha"] = (1.0 / (a_gs * w_gs)).reshape(1).expand(1 if op == "epilogue" else 2).contiguous()
    s["bias"] = _bf16(g, N, std=0.5) if case["bias"] else None
    s["res"] = _bf16(g, M, N, std=2.0) if case.get("residual") else None
    s["d"] = torch.empty(M, cols, dtype=torch.bfloat16, device=DEV)
    s["ws"] = torch.zeros(WORKSPACE, dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------ the plain form

def _values(codes, sf):
    """NVFP4 codes and scale bytes -> fp32 values."""
    grid = torch.tensor(CODES + tuple(-v for v in CODES), device=codes.device)
    pair = torch.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1)
    v = grid[pair.int()].reshape(codes.shape[0], -1, 16)
    return (v * sf.view(torch.float8_e4m3fn).float()[..., None]).reshape(codes.shape[0], -1)


def _act(x, act):
    if act == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if act == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    return x


def _norm(x, w, b, kind):
    d = x.double()
    if kind == LAYER:
        d = d - d.mean(-1, keepdim=True)
    rstd = (1.0 / torch.sqrt((d * d).mean(-1, keepdim=True) + 1e-6)).float()
    y = d.float() * rstd * w.float()
    return y if b is None else y + b.float()


def _plain_epilogue(s):
    v = _values(s["a"], s["a_sf"]) @ _values(s["w"], s["w_sf"]).t() * s["alpha"]
    if s["bias"] is not None:
        v = v + s["bias"].float()
    v = _act(v, s["act"])
    if s["res"] is not None:
        v = v + s["res"].float()
    return v.to(torch.bfloat16)


def _plain_gated(s):
    v = _values(s["a"], s["a_sf"]) @ _values(s["w"], s["w_sf"]).t()
    I = s["I"]
    gate, up = v[:, :I] * s["alpha"][0], v[:, I:] * s["alpha"][1]
    if s["bias"] is not None:
        gate, up = gate + s["bias"][:I].float(), up + s["bias"][I:].float()
    return (_act(gate, s["act"]) * up).to(torch.bfloat16)


def _plain_norm(s):
    u = s["x"].float()
    if s["post"]:
        u = _norm(u, s["pw"], s["pb"], s["kind"])
    if s["g"] is not None:
        gate = s["g"].float()
        if s["gate"] > 0:
            gate = gate.repeat_interleave(s["gate"], 0)[: s["T"]]
        u = gate * u
    r = s["res"].float() + u
    return [r.to(torch.bfloat16), _norm(r, s["w"], s["b"], s["kind"]).to(torch.bfloat16)]


def _plain_block(s):
    I = s["I"]
    r = s["res"].float() + s["x"].float()
    r16 = r.to(torch.bfloat16)
    q, sf = _quantize(_norm(r, s["w"], None, RMS), s["gs_x"])
    y = (q.reshape(-1, 16) * sf.float().reshape(-1, 1)).reshape(q.shape)
    gu = y @ _values(s["gu"], s["gu_sf"]).t()
    h = _act(gu[:, :I] * s["alpha_gu"][0], "silu") * (gu[:, I:] * s["alpha_gu"][1])
    q, sf = _quantize(h, s["gs_h"])
    h = (q.reshape(-1, 16) * sf.float().reshape(-1, 1)).reshape(q.shape)
    d = h @ _values(s["dn"], s["dn_sf"]).t() * s["alpha_dn"] + r16.float()
    return [r16, d.to(torch.bfloat16)]


# ------------------------------------------------------- the library's calls

def _own(s):
    import nvfp4_block_scaled_07_amd as nv
    op = s["op"]
    if op == "epilogue":
        return nv.nvfp4_gemm_epilogue(s["a"], s["a_sf"], s["w"], s["w_sf"], s["alpha"], s["bias"], ACTS[s["act"]],
                                      s["res"], 1.0, s["d"], s["M"], s["N"], s["K"], s["ws"])
    if op == "gated":
        return nv.nvfp4_gemm_gated(s["a"], s["a_sf"], s["w"], s["w_sf"], s["alpha"], s["bias"], ACTS[s["act"]],
                                   s["d"], s["M"], s["I"], s["K"], s["ws"])
    if op == "norm":
        nv.nvfp4_residual_norm(s["x"], s["pw"], s["pb"], s["g"], max(s["gate"], 0), s["res"], 1.0, s["w"], s["b"],
                               1e-6, s["kind"], s["r"], s["y"], None, None, None, s["T"], s["H"])
        return [s["r"], s["y"]]
    M, H, I = s["M"], s["H"], s["I"]
    nv.nvfp4_residual_norm(s["x"], None, None, None, 0, s["res"], 1.0, s["w"], None, 1e-6, RMS, s["r"], None,
                           s["gs_x"], s["q"], s["sf"], M, H)
    nv.nvfp4_ffn(s["q"], s["sf"], s["gu"], s["gu_sf"], s["alpha_gu"], None, ACTS["silu"], s["gs_h"], s["dn"],
                 s["dn_sf"], s["alpha_dn"], None, s["r"], 1.0, s["d"], M, H, I, s["ws"])
    return [s["r"], s["d"]]


_PLAIN = {"epilogue": _plain_epilogue, "gated": _plain_gated, "norm": _plain_norm, "block": _plain_block}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------------------ 64 bits

def _decode64(codes, sf):
    """Values of NVFP4 codes and e4m3 bytes from the formats' fields, in 64 bits."""
    low = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.uint8, device=codes.device)
    low[:, 0::2], low[:, 1::2] = codes & 0xF, codes >> 4
    mag, man = (low >> 1) & 3, (low & 1).double()
    v = torch.where(mag == 0, man * 0.5, (1.0 + man / 2) * torch.exp2(mag.double() - 1))
    v = torch.where(low >= 8, -v, v)
    e, m = (sf >> 3) & 15, (sf & 7).double()
    scale = torch.where(e == 0, m * 2.0 ** -9, (1.0 + m / 8) * torch.exp2(e.double() - 7))
    return v * scale.repeat_interleave(16, 1)


def _round_nvfp4_64(x, gs):
    """The values that the NVFP4 quantisation of x (fp64, encode scale gs) stands for, times gs."""
    rows, K = x.shape
    peak = x.abs().reshape(rows, K // 16, 16).amax(-1)
    t = torch.clamp(peak / 6.0 * gs, max=448.0)
    grain = torch.exp2(torch.clamp(torch.floor(torch.log2(torch.clamp(t, min=2.0 ** -30))), min=-6.0) - 3.0)
    scale = torch.round(t / grain) * grain
    inv = torch.where(scale > 0, gs / scale, torch.zeros_like(scale)).repeat_interleave(16, 1)
    v = x * inv
    below = 1.0 - 2.0 ** -52  # ties go to the even code: up at 0.75, 1.75 and 3.5
    edges = torch.tensor([0.25, 0.75 * below, 1.25, 1.75 * below, 2.5, 3.5 * below, 5.0], dtype=torch.float64,
                         device=x.device)
    mag = torch.tensor(CODES, dtype=torch.float64, device=x.device)[torch.bucketize(v.abs(), edges)]
    return torch.sign(v) * mag * scale.repeat_interleave(16, 1)


def _act64(x, act):
    if act == "relu":
        return torch.clamp(x, min=0.0)
    if act == "gelu":
        return x * torch.special.ndtr(x)
    if act == "gelu_tanh":
        z = 2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3)
        return x * torch.sigmoid(z)
    if act == "silu":
        return x * torch.sigmoid(x)
    return x


def _norm64(x, w, b, kind):
    mean = x.mean(-1, keepdim=True) if kind == LAYER else 0.0
    var = ((x - mean) ** 2).sum(-1, keepdim=True) / x.shape[-1]
    y = (x - mean) / torch.sqrt(var + 1e-6) * w.double()
    return y + b.double() if b is not None else y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        u = s["x"].double()
        if s["pw"] is not None:
            u = _norm64(u, s["pw"], s["pb"], case["kind"])
        if s["g"] is not None:
            rows = torch.arange(case["T"], device=DEV) // max(case["gate"], 1) if case["gate"] > 0 else None
            u = u * (s["g"].double() if rows is None else s["g"].double()[rows])
        r = u + s["res"].double()
        return [r, _norm64(r, s["w"], s["b"], case["kind"])]
    if op == "block":
        I = case["I"]
        r = s["x"].double() + s["res"].double()
        y = _round_nvfp4_64(_norm64(r, s["w"], None, RMS), s["gs_x"].double())
        gu = y @ _decode64(s["gu"], s["gu_sf"]).t()
        h = _act64(gu[:, :I] * s["alpha_gu"][0].double(), "silu") * (gu[:, I:] * s["alpha_gu"][1].double())
        h = _round_nvfp4_64(h, s["gs_h"].double())
        d = h @ _decode64(s["dn"], s["dn_sf"]).t() * s["alpha_dn"].double()
        # the stream that the block's output is added to is held in bf16
        return [r, d + r.to(torch.bfloat16).double()]
    v = _decode64(s["a"], s["a_sf"]) @ _decode64(s["w"], s["w_sf"]).t()
    if op == "epilogue":
        v = v * s["alpha"].double()
        v = _act64(v + s["bias"].double() if s["bias"] is not None else v, case["act"])
        return v + s["res"].double() if s["res"] is not None else v
    I = case["I"]
    gate, up = v[:, :I] * s["alpha"][0].double(), v[:, I:] * s["alpha"][1].double()
    if s["bias"] is not None:
        gate, up = gate + s["bias"][:I].double(), up + s["bias"][I:].double()
    return _act64(gate, case["act"]) * up
