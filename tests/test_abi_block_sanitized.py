"""The host layer of the block operators under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only): the library with the sanitizers on its
host code, linked with tests/abi_block_sanitize.cpp, which walks plan choice,
workspace sizes and refusals; any report aborts the run and no kernel is
launched."""
import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from nvfp4_block_scaled_07_amd import build as b
from tests.test_abi_sanitized import CLANG, HIPCC, HOST_SAN, ROCM, ROOT, _run


@pytest.mark.timeout(900)
def test_block_operators_under_address_and_undefined_behaviour_sanitizers(tmp_path):
    if not (os.path.exists(HIPCC) and os.path.exists(CLANG)):
        pytest.skip("the ROCm compilers are not installed")
    objs, cmds = [], []
    for src in [*b.SOURCES, *b.SCHED_SOURCES, *b.BLOCK_SOURCES]:
        objs.append(str(tmp_path / (os.path.splitext(os.path.basename(src))[0] + ".o")))
        # device code as quickly as it compiles: it is never launched
        cmds.append([HIPCC, "--offload-arch=gfx950", "-std=c++17", "-O1", "-g", "-Xclang", "-target-feature", "-Xclang",
                     "-packed-fp32-ops", *HOST_SAN, "-I", os.path.join(ROOT, "include"), "-c", os.path.join(b.CSRC, src),
                     "-o", objs[-1]])
    drv = str(tmp_path / "driver.o")
    cmds.append([CLANG, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-I",
                 os.path.join(ROOT, "include"), "-c", os.path.join(ROOT, "tests", "abi_block_sanitize.cpp"), "-o", drv])
    with ThreadPoolExecutor(8) as ex:
        list(ex.map(_run, cmds))
    exe = str(tmp_path / "abi_block_sanitize")
    _run([CLANG, "-fsanitize=address,undefined", *objs, drv, f"-L{ROCM}/lib", "-lamdhip64", f"-Wl,-rpath,{ROCM}/lib", "-o", exe])
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    run = subprocess.run([exe], capture_output=True, text=True, env=env, timeout=600)
    out = run.stdout + run.stderr
    assert run.returncode == 0, out[-4000:]
    assert "all host checks passed" in run.stdout
    assert "runtime error" not in out and "AddressSanitizer" not in out
