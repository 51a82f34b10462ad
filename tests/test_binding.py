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
