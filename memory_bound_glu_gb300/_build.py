"""Builds libmbglu.so in-tree with nvcc for sm_103a (GB300).

No fast math (DeepSpeed PR #9057 "Changes" removed --use_fast_math from the
fused-GLU build): expf and division keep their IEEE-accurate forms.
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libmbglu.so")
QUICK = os.path.join(HERE, "_mbglu_torch.so")   # the binding's extension module
SOURCES = [os.path.join(HERE, "csrc", f) for f in ("mbglu_api.cu", "gemm_api.cu", "fp8_api.cu")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    # share the process's CUDA runtime (the one torch loads), so the current
    # device and streams are one state; rpath for standalone C callers
    "-cudart", "shared", "-Xlinker", "-rpath,/usr/local/cuda/lib64",
    "-I", os.path.join(ROOT, "include"),
]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def quick_stamp() -> str:
    """What the extension module is built against: it fits no other torch or Python."""
    import torch
    return f"built for torch {torch.__version__}, {sys.implementation.cache_tag}"


def quick_is_current() -> bool:
    """Whether the extension module is there and fits the torch that is installed: its
    description says what it was built against."""
    try:
        with open(QUICK, "rb") as f:
            return quick_stamp().encode() + b"\0" in f.read()
    except OSError:
        return False


def _sources_and_headers():
    csrc = os.path.join(HERE, "csrc")
    return [os.path.join(csrc, f) for f in sorted(os.listdir(csrc))] + [os.path.join(ROOT, "include", "mbglu.h")]


def needs_build(out: str = LIB) -> bool:
    if not os.path.exists(out) or not quick_is_current():
        return True
    t = min(os.path.getmtime(out), os.path.getmtime(QUICK))
    return any(os.path.getmtime(f) > t for f in _sources_and_headers())


def build_quick() -> str:
    """The binding's extension module, against the torch that is installed."""
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    inc = [os.path.join(ROOT, "include"), os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include"),
           os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"]]
    if os.path.exists(QUICK):   # a failing build leaves no old module behind
        os.remove(QUICK)
    subprocess.run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
                    f'-DMBGLU_BUILT_FOR="{quick_stamp()}"',
                    f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f for i in inc for f in ("-I", i)),
                    "-o", QUICK, os.path.join(HERE, "csrc", "bind_torch.cpp"), "-L", os.path.join(base, "lib"),
                    "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"], check=True)
    return QUICK


def build(out: str = LIB, verbose: bool = False, extra=()) -> str:
    """Compiles the translation units in parallel, then links them; beside
    them the binding's extension module.  That one needs Python's and torch's
    headers and a CUDA build of torch, the library none of them: where the module
    cannot be built, a warning says so and binding.py does without it."""
    compile_flags = [f for f in NVCC_FLAGS if f != "-shared"]

    def one(src, obj):
        cmd = [nvcc(), *compile_flags, *extra, "-c", "-o", obj, src]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        subprocess.run(cmd, check=True)

    with tempfile.TemporaryDirectory() as tmp:
        objs = [os.path.join(tmp, os.path.basename(s) + ".o") for s in SOURCES]
        with ThreadPoolExecutor(len(SOURCES) + 1) as ex:
            quick = ex.submit(build_quick)
            for f in [ex.submit(one, s, o) for s, o in zip(SOURCES, objs)]:
                f.result()
        subprocess.run([nvcc(), *NVCC_FLAGS, "-o", out, *objs], check=True)
    try:
        quick.result()
    except Exception as e:
        warnings.warn(f"the binding's extension module was not built ({e}): the wide and the e4m3 calls take 10 to 15 us "
                      "more of host time")
    return out


if __name__ == "__main__":
    build(verbose="-v" in sys.argv)
    print(LIB)
