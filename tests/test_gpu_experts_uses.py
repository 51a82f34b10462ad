"""Calls of the mixture-of-experts operators that their documentation allows and
that belong to no operator's own tests."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_07_amd as nv
from tests.experts_util import dev_mx, mx_operand, offsets_of, out_bytes
from tests.gpu_util import dev, host, say

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
