"""The workspace helpers zero-fill on the GPU that holds the workspace, on its
current stream (CPU only: the GPUs are stand-ins)."""
from types import SimpleNamespace

import pytest
import torch

import nvfp4_block_scaled_07_amd as nv


class Library:
    """The library with its zero-fill recorded instead of launched."""

    def __init__(self, real, gpus):
        self._real, self._gpus, self.fills = real, gpus, []

    def __getattr__(self, name):
        return getattr(self._real, name)

    def nvfp4_workspace_init(self, ptr, nbytes, stream):
        self.fills.append((self._gpus.current, stream.value, nbytes))
        return 0


class Workspace:
    is_cuda = True

    def __init__(self, n, device):
        self.n, self.device = n, torch.device(device)

    def is_contiguous(self):
        return True

    def numel(self):
        return self.n

    def element_size(self):
        return 1

    def data_ptr(self):
        return 0x10000


@pytest.fixture
def library(monkeypatch):
    gpus = SimpleNamespace(current=0)

    class device:
        def __init__(self, d):
            self.to = torch.device(d).index

        def __enter__(self):
            self.before, gpus.current = gpus.current, self.to

        def __exit__(self, *e):
            gpus.current = self.before
            return False
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: SimpleNamespace(cuda_stream=1000 + gpus.current))
    monkeypatch.setattr(torch, "empty", lambda n, dtype, device: Workspace(n, device))
    lib = Library(nv.lib(), gpus)
    monkeypatch.setattr(nv, "_lib", lib)
    yield lib
    assert gpus.current == 0


@pytest.mark.parametrize("make,shape", [(nv.gemm_epilogue_workspace, (1024, 768, 6144)), (nv.gemm_gated_workspace, (16, 2048, 6144)),
                                        (nv.ffn_workspace, (16, 512, 256)), (nv.gemm_workspace, (512, 768, 6144))])
def test_zero_filled_where_it_lies(library, make, shape):
    ws = make(*shape, device="cuda:1")
    make(*shape, device="cuda:0")
    assert library.fills == [(1, 1001, ws.n), (0, 1000, ws.n)]


def test_a_given_stream_is_kept(library):
    nv.nvfp4_workspace_init(Workspace(4096, "cuda:2"), stream=77)
    assert library.fills == [(2, 77, 4096)]
