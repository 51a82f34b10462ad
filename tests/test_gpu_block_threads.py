"""Block operators called by several Python threads at once, each on a stream
and a workspace of its own: the calls do not hold the interpreter lock, so they
really overlap on the host."""
import threading

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_07_amd as nv
from tests.block_util import bf16, dev_bf16, operand
from tests.gpu_util import dev, scalar

pytestmark = pytest.mark.gpu


def _layer(seed, M, H, I):
    """The norm and the feed-forward of one thread, and a fresh output to run them into."""
    rng = np.random.default_rng(seed)
    (gu, gusf, _), (dn, dnsf, _) = operand(seed, 2 * I, H), operand(seed + 2, H, I)
    x, w = dev_bf16(bf16(rng.standard_normal((M, H)))), dev_bf16(bf16(rng.standard_normal(H) * 0.1 + 1))
    q, sf = torch.empty(M, H // 2, dtype=torch.uint8, device="cuda"), torch.empty(M, H // 16, dtype=torch.uint8, device="cuda")
    r, d = torch.empty_like(x), torch.empty_like(x)
    weights = dev(gu), dev(gusf), dev(np.array([1e-3, 1e-3], np.float32)), None, nv.ACT_SILU, scalar(50.0), dev(dn), dev(dnsf), scalar(1e-4), None
    gs, ws = scalar(300.0), nv.ffn_workspace(M, H, I)

    def run():
        nv.nvfp4_residual_norm(x, None, None, None, 0, x, 1.0, w, None, 1e-6, nv.NORM_RMS, r, None, gs, q, sf, M, H)
        return nv.nvfp4_ffn(q, sf, *weights, r, 1.0, d, M, H, I, ws)
    return run


@pytest.mark.timeout(120)
def test_threads_on_streams_of_their_own():
    # a split gated product, unsplit register tiles, LDS tiles, and a refusal in a thread of its own
    layers = [_layer(10, 16, 6144, 2048), _layer(20, 1, 512, 256), _layer(30, 300, 512, 1024)]
    want = [run().clone() for run in layers]
    torch.cuda.synchronize()
    wrong, errors = [], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for n in range(30):
                    d = layers[i]()
                    if n % 10 == 9:
                        torch.cuda.current_stream().synchronize()
                        if not torch.equal(d, want[i]):
                            wrong.append((i, n))
        except Exception as e:  # told by the test, not by the thread
            errors.append(e)

    def refused():
        for _ in range(200):
            with pytest.raises(nv.Nvfp4Error) as e:
                nv.nvfp4_gemm_gated(None, None, None, None, None, None, 9, None, 1, 16, 256)
            if "act = 9" not in str(e.value):
                errors.append(e.value)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)] + [threading.Thread(target=refused)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and not wrong, (errors, wrong)
