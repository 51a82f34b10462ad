"""nvfp4_moe_sort against the oracle: whole numbers, equal."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_07_amd as nv
from oracle import experts_ref as x
from tests.gpu_util import dev, host, say

pytestmark = pytest.mark.gpu


def run(ids, first, E):
    T, k = ids.shape
    off = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda")
    tok = torch.full((max(T * k, 1),), -7, dtype=torch.int32, device="cuda")
    rows = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    ws = nv.moe_sort_workspace(T, E, k)
    if ws is not None:
        ws.fill_(0xA5)
    nv.nvfp4_moe_sort(ids, first, off, tok, rows, T, E, k, ws)
    return host(off), host(tok), host(rows)


def fast(ids, first, E):
    """sort_rows by numpy's stable sort, for many rows."""
    e = ids.reshape(-1).astype(np.int64) - first
    inside = (e >= 0) & (e < E)
    order = np.argsort(np.where(inside, e, E), kind="stable")[:int(inside.sum())]
    rows = np.full(ids.size, -1, np.int32)
    rows[order] = np.arange(order.size)
    return np.searchsorted(e[order], np.arange(E + 1)).astype(np.int32), (order // ids.shape[1]).astype(np.int32), rows.reshape(ids.shape)


def check(ids, first, E, oracle):
    off, tok, rows = run(dev(ids), first, E)
    want = oracle(ids, first, E)
    np.testing.assert_array_equal(off, want[0])
    np.testing.assert_array_equal(rows, want[2])
    n = int(off[-1])
    np.testing.assert_array_equal(tok[:n], want[1])
    assert (tok[n:] == -7).all()  # rows that no expert has stay as they were


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (3, 5, 2), (61, 60, 4), (64, 8, 8), (100, 300, 7), (513, 17, 3)])
def test_small_against_the_oracle(T, E, k):
    say("sort", T, E, k)
    rng = np.random.default_rng(T + E)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)  # a token may name an expert twice
    check(ids, 0, E, x.sort_rows)
    check(ids, 0, max(1, E // 2), x.sort_rows)            # the others are left out
    check(ids, E // 3, max(1, E // 3), x.sort_rows)
    wild = ids.copy()
    wild.reshape(-1)[:: 3] = rng.choice([-1, E, 2 ** 31 - 1, -2 ** 31], wild.reshape(-1)[:: 3].shape)
    check(wild, 0, E, x.sort_rows)


@pytest.mark.parametrize("T,E,k", [(1023, 64, 1), (4097, 256, 8), (16384, 256, 8), (33333, 7, 6), (50001, 1000, 9),
                                   (200000, 128, 8)])
def test_many_rows(T, E, k):
    say("sort", T, E, k)
    rng = np.random.default_rng(T)
    ids = np.minimum((rng.random((T, k)) ** 2 * (E + 3)).astype(np.int32), E)  # uneven, some outside
    np.testing.assert_array_equal(fast(ids[:50], 0, E)[2], x.sort_rows(ids[:50], 0, E)[2])
    check(ids, 0, E, fast)
    check(np.full((T, k), E - 1, np.int32), 0, E, fast)  # one expert has all


def test_many_experts():
    # above 1024 experts the form for few ids takes more of them, too
    ids = np.random.default_rng(5).integers(-2, 1505, (9000, 6)).astype(np.int32)
    check(ids, 0, 1500, fast)
    check(ids[:10], 3, 65535, fast)


def test_wild_ids_among_many():
    rng = np.random.default_rng(6)
    ids = rng.integers(0, 40, (9000, 6)).astype(np.int32)
    ids.reshape(-1)[::5] = rng.choice([-1, 40, 64, 2 ** 31 - 1, -2 ** 31, -2 ** 31 + 7], ids.reshape(-1)[::5].shape)
    check(ids, 0, 40, fast)
    check(ids, 7, 20, fast)


def test_no_rows():
    for T, k in ((0, 8), (5, 0)):
        off, tok, _ = run(torch.empty(T, k, dtype=torch.int32, device="cuda"), 0, 6)
        assert (off == 0).all() and (tok == -7).all()


def test_captured_and_replayed():
    for T, E, k in ((40, 32, 4), (30000, 64, 8)):
        g = torch.Generator(device="cuda").manual_seed(T)
        ids = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda", generator=g)
        off, tok, rows = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (E + 1, T * k, T * k))
        ws = nv.moe_sort_workspace(T, E, k)
        args = (ids, 0, off, tok, rows, T, E, k, ws)
        nv.nvfp4_moe_sort(*args)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            nv.nvfp4_moe_sort(*args)
        for _ in range(3):
            ids.copy_(torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda", generator=g))
            graph.replay()
            torch.cuda.synchronize()
            want = fast(host(ids), 0, E)
            for got, w in zip((off, tok, rows), want):
                np.testing.assert_array_equal(host(got), w.reshape(-1))


def test_refused_tensors():
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    off, tok, rows = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (9, 8, 8))
    nv.nvfp4_moe_sort(ids, 0, off, tok, rows, 4, 8, 2)
    for bad in ((ids.long(), 0, off, tok, rows, 4, 8, 2), (ids, 0, off[:8], tok, rows, 4, 8, 2),
                (ids, 0, off, tok[:7], rows, 4, 8, 2), (ids, 0, off, tok, rows[:7], 4, 8, 2),
                (ids, 0, off, tok, rows, 5, 8, 2), (ids.t(), 0, off, tok, rows, 4, 8, 2),
                (ids, -1, off, tok, rows, 4, 8, 2), (ids.cpu(), 0, off, tok, rows, 4, 8, 2)):
        with pytest.raises(nv.Nvfp4Error):
            nv.nvfp4_moe_sort(*bad)
