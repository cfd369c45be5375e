"""Build step of the C-ABI library: nvcc for sm_103a, one object per .cu in
parallel, linked into ``libgdn.so`` inside the package directory (in-tree), and
of the binding's argument marshalling, ``_binding.<torch>.<python>.so`` beside it
(g++, against torch's headers).

No fast-math flags: the kernels rely on IEEE division, expf/log1pf and
explicit round-to-nearest adds and multiplies.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libgdn.so")
SOURCES = ["gdn_api.cu", "gdn_conv.cu", "gdn_decode.cu", "gdn_prefill.cu", "gdn_prefill_tc.cu",
           "gdn_graph.cu", "gdn_noalloc.cu", "gdn_gate.cu", "gdn_mixed.cu",
           "gdn_cache_api.cu", "gdn_cache.cu", "gdn_attn_decode.cu",
           "gdn_attn_prefill.cu", "gdn_rope.cu", "gdn_cache4.cu", "gdn_attn4_decode.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE]


def _nvcc() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(home, "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "gdn.h"))
    return files


def binding_path() -> str:
    """The binding links torch's C++ libraries and Python's: its name says which, so another version finds none of its own."""
    import torch

    return os.path.join(PKG, f"_binding.{torch.__version__}.{sysconfig.get_config_var('SOABI')}.so")


def stale(binding: bool = True) -> bool:
    built = [LIB, binding_path()] if binding else [LIB]
    if not all(os.path.exists(f) for f in built):
        return True
    t = min(os.path.getmtime(f) for f in built)
    return any(os.path.getmtime(f) > t for f in _inputs())


def _binding_command(out: str) -> list[str]:
    import torch

    home = os.path.dirname(torch.__file__)
    lib = os.path.join(home, "lib")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    include = [INCLUDE, os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={abi}", *("-I" + i for i in include),
            os.path.join(CSRC, "gdn_binding.cpp"), "-o", out, "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
            "-Wl,-rpath," + lib]


def _finish(procs) -> str:
    """What the commands that failed wrote; empty if none did."""
    failed = []
    for cmd, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append(" ".join(cmd) + "\n" + out.decode(errors="replace"))
    return "\n".join(failed)


def build_library(force: bool = False, verbose: bool = False, binding: bool = True) -> str:
    """Compile every CUDA source for sm_103a, link libgdn.so and compile the binding (skipped when up to date). The library
    stands by itself: where the binding does not compile, it is linked all the same before that is raised. binding=False
    leaves the binding out, for users of the C ABI without torch's and Python's headers."""
    try:
        if not force and not stale(binding):
            return LIB
    except ImportError:  # no torch: the library at least
        pass
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()

    def start(cmd):
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        return cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)

    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        objs.append(obj)
        procs.append(start([nvcc, *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]))
    binding_procs, no_binding, tmp_binding = [], "", ""
    if binding:
        try:
            tmp_binding = binding_path() + f".tmp{os.getpid()}"
            binding_procs.append(start(_binding_command(tmp_binding)))
        except (ImportError, OSError) as e:  # no torch, or no g++
            no_binding = repr(e)
    msg = _finish(procs)
    if not msg:
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.check_call([nvcc, *ARCH, "-shared", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    no_binding = no_binding or _finish(binding_procs)
    if msg:
        if os.path.exists(tmp_binding):
            os.remove(tmp_binding)
        raise RuntimeError("nvcc failed:\n" + msg)
    if no_binding:
        raise RuntimeError(f"{LIB} is built, its binding for Python failed:\n" + no_binding)
    if binding:
        os.replace(tmp_binding, binding_path())
    return LIB


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose=True, binding="--library" not in sys.argv))
