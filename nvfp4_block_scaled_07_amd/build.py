"""Build the gfx950 shared library ``libnvfp4_gfx950.so`` in-tree with hipcc.

Run ``python -m nvfp4_block_scaled_07_amd.build`` (or call :func:`build`).
The quantiser needs IEEE fp32 semantics, so there is no fast-math, fp
contraction is off and fp32 division stays correctly rounded.  Packed fp32
instructions are disabled for all device code.  ``gemm_large.hip`` (the two
large-M NVFP4 tiles) is compiled to an object of its own, with the iterative
ILP instruction scheduler, and so is each source of the block operators
(``csrc/block``), all at the same time as the rest; one last hipcc call links
them.  ``csrc/binding.cpp``, the native marshalling of the block operators'
Python calls, is host code against torch's headers and becomes ``_binding``
(with the interpreter's suffix); the library does not depend on it.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libnvfp4_gfx950.so")
# named for the interpreter it is compiled for, so that another one does not load it
BINDING = os.path.join(PKG, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
SOURCES = ["api.hip", "gemm.hip", "layout.hip", "moe.hip", "quantize.hip"]
# sources compiled separately, with extra flags
SCHED_SOURCES = {"gemm_large.hip": ["-mllvm", "-amdgpu-sched-strategy=iterative-ilp"]}
# the block operators, each source an object of its own, with its extra flags
BLOCK_SOURCES = {
    "block/block_api.hip": [],
    "block/norm.hip": [],
    "block/gemm_epilogue.hip": [],
    "block/gemm_epilogue_large.hip": ["-mllvm", "-amdgpu-sched-strategy=iterative-ilp"],
}
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-ffp-contract=off", "-fno-fast-math", "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-Wall", "-Wno-unused-command-line-argument",
    "-I", os.path.join(ROOT, "include"),
]


def _object(objdir: str, src: str) -> str:
    return os.path.join(objdir, os.path.splitext(os.path.basename(src))[0] + ".o")


def object_commands(objdir: str) -> list:
    """hipcc calls that compile every source to an object in objdir."""
    flags = [f for f in FLAGS if f != "-shared"]
    sources = {**{s: [] for s in SOURCES}, **SCHED_SOURCES, **BLOCK_SOURCES}
    return [[HIPCC, *flags, *extra, "-c", os.path.join(CSRC, src), "-o", _object(objdir, src)]
            for src, extra in sources.items()]


def command(out: str = LIB, objdir: str = "") -> list:
    """The hipcc call that links the objects in objdir."""
    objs = [_object(objdir, s) for s in [*SOURCES, *SCHED_SOURCES, *BLOCK_SOURCES]]
    return [HIPCC, *FLAGS, *objs, "-o", out]


def binding_command(out: str = BINDING) -> list:
    """The g++ call that compiles the marshalling module against torch's headers."""
    import torch
    t = os.path.dirname(os.path.abspath(torch.__file__))
    rocm = os.path.dirname(os.path.dirname(HIPCC))
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
            "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM", f'-DNVFP4_TORCH_VERSION="{torch.__version__}"', f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-isystem", os.path.join(t, "include"), "-isystem", os.path.join(rocm, "include"),
            "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, "binding.cpp"), "-o", out,
            "-L", os.path.join(t, "lib"), "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_python"]


def _run(cmd: list, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    try:
        res = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError(f"{cmd[0]} cannot be run: {e}") from e
    # the host pass warns about the device-only target feature; that is harmless
    msgs = [l for l in (res.stdout + res.stderr).splitlines()
            if l.strip() and "packed-fp32-ops" not in l and "is not a recognized feature" not in l]
    if res.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed:\n" + "\n".join(msgs))
    if verbose and msgs:
        print("\n".join(msgs))


def _remove(path: str) -> None:
    if os.path.exists(path):
        os.remove(path)


def build(verbose: bool = False) -> str:
    """Compile every HIP source into the in-tree library, and the marshalling
    module; returns the library's path.

    The library needs neither torch nor a host compiler: it is in place whatever
    becomes of the module, which is left out (with a note) without torch, and
    whose own failure is raised afterwards.  A module of an earlier build never
    stays beside a newer library."""
    tmp, btmp = LIB + ".tmp", BINDING + ".tmp"
    try:
        module = binding_command(btmp)
    except ImportError as e:
        module = None
        print(f"{os.path.basename(BINDING)} is left out, the Python calls of the block operators need it: {e}", file=sys.stderr)
    try:
        with tempfile.TemporaryDirectory(prefix="nvfp4_build_") as objdir:
            with ThreadPoolExecutor(len(os.sched_getaffinity(0))) as pool:
                objects = [pool.submit(_run, cmd, verbose) for cmd in object_commands(objdir)]
                binding = pool.submit(_run, module, verbose) if module else None
            for done in objects:
                done.result()
            _run(command(tmp, objdir), verbose)
        _remove(BINDING)
        os.replace(tmp, LIB)
        if binding:
            binding.result()
            os.replace(btmp, BINDING)
    finally:
        _remove(tmp)
        _remove(btmp)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
