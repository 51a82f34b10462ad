"""The native marshalling module of the block operators on the CPU: what it
does around the library's call."""
import ctypes
import shutil
import subprocess
import threading

import pytest

import nvfp4_block_scaled_07_amd as nv

# stands in for a launch that waits for queue space: done when another Python thread has run
WAITING_CALL = r"""
#include <unistd.h>
volatile int entered = 0, other_ran = 0;
int waiting_call(void) {
  entered = 1;
  for (int i = 0; i < 2000 && !other_ran; ++i) usleep(1000);
  return other_ran ? 0 : 6;
}
const char* message(void) { return "no other thread ran"; }
"""


@pytest.mark.timeout(60)
def test_other_threads_run_during_a_call(tmp_path):
    cc = shutil.which("cc") or shutil.which("gcc") or shutil.which("g++")
    if not cc:
        pytest.skip("no C compiler")
    src, so = tmp_path / "waiting.c", str(tmp_path / "waiting.so")
    src.write_text(WAITING_CALL)
    subprocess.run([cc, "-O1", "-shared", "-fPIC", "-x", "c", str(src), "-o", so], check=True)
    c = ctypes.CDLL(so)
    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value
    entered, ran = ctypes.c_int.in_dll(c, "entered"), ctypes.c_int.in_dll(c, "other_ran")
    binding = nv._native()

    def other():
        while not entered.value:
            pass
        ran.value = 1
    t = threading.Thread(target=other, daemon=True)
    try:
        binding.setup(nv.Nvfp4Error, address(c.message), *[address(c.waiting_call)] * 5)
        t.start()
        nv.nvfp4_residual_norm(None, None, None, None, 0, None, 1.0, None, None, 1e-6, 0, None, None, None, None, None, 0, 64)
    finally:
        entered.value = 1
        nv._bind = None
        nv._native()  # bound to the library again
    t.join()
    # and a refusal's message is still the calling thread's
    with pytest.raises(nv.Nvfp4Error) as e:
        nv.nvfp4_residual_norm(None, None, None, None, 0, None, 1.0, None, None, 1e-6, 0, None, None, None, None, None, 0, 0)
    assert e.value.status == 2 and "H = 0" in str(e.value)


def _native_error(monkeypatch, package_dir):
    """The ImportError of loading the module from package_dir."""
    import sys
    monkeypatch.setattr(nv, "_bind", None)
    monkeypatch.setattr(nv, "__path__", [str(package_dir)])
    monkeypatch.delattr(nv, "_binding", raising=False)
    monkeypatch.delitem(sys.modules, "nvfp4_block_scaled_07_amd._binding", raising=False)
    with pytest.raises(ImportError) as e:
        nv._native()
    return str(e.value)


def test_a_missing_module_and_one_that_does_not_load_are_told_apart(tmp_path, monkeypatch):
    text = _native_error(monkeypatch, tmp_path)
    assert "is missing" in text and "nvfp4_block_scaled_07_amd.build" in text
    (tmp_path / "_binding.so").write_bytes(b"not a shared object")
    text = _native_error(monkeypatch, tmp_path)
    assert "is missing" not in text and "nvfp4_block_scaled_07_amd.build" in text
    assert "invalid ELF header" in text or "too short" in text  # the loader's own words


def test_a_module_built_for_another_torch_is_refused(monkeypatch):
    import os

    import torch
    here = os.path.dirname(nv.__file__)
    monkeypatch.setattr(torch, "__version__", "1.0.0+other")
    text = _native_error(monkeypatch, here)
    assert "1.0.0+other" in text and "nvfp4_block_scaled_07_amd.build" in text
    monkeypatch.undo()
    assert nv._native() is not None
