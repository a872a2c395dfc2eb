"""Builds the in-tree CUDA library ``libfa_gb300.so`` for sm_103a.

Each ``csrc/*.cu`` translation unit is compiled by ``nvcc`` in parallel, then
linked into one shared library beside this file. Only a CUDA toolkit with
sm_103a support is needed (the build cross-compiles without a GPU). Where
PyTorch with CUDA is installed, ``csrc/fa_calls.cpp`` is built beside them as
the Python module ``_calls`` against its headers. The library does without
that module: where it cannot be built, the build says so and goes on.

Usage: ``python -m exact_attention_80_gb300.build [--ptxas-verbose]``
"""

from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfa_gb300.so")
CALLS = os.path.join(PKG, "_calls.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: a CUDA 13 toolkit is required to build libfa_gb300.so")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _compile(nvcc: str, src: str, ptxas_verbose: bool) -> tuple[str, str]:
    obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc, *ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-c", src, "-o", obj]
    if ptxas_verbose:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stdout + r.stderr


def build_calls() -> str | None:
    """Compile ``csrc/fa_calls.cpp`` into the module ``_calls``. None, and no module left from an earlier
    build, where there is no PyTorch with CUDA or the module does not compile against it."""
    if os.path.exists(CALLS):
        os.remove(CALLS)
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    torch = spec.submodule_search_locations[0]
    if not os.path.exists(os.path.join(torch, "lib", "libc10_cuda.so")):
        return None
    with open(os.path.join(torch, "version.py"), encoding="utf-8") as f:
        version = re.search(r"^__version__ *(?::.*?)?= *['\"](.*?)['\"]", f.read(), re.M)
    version = version.group(1) if version else "an unknown version"  # (which the binding will not take)
    inc, tmp = os.path.join(torch, "include"), CALLS + ".tmp"
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    cmd = [shutil.which("g++") or "g++", "-std=c++17", "-O2", "-fPIC", "-shared", f'-DFA_TORCH_VERSION="{version}"',
           "-I", os.path.join(ROOT, "include"), "-I", sysconfig.get_paths()["include"], "-isystem", inc,
           "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), os.path.join(CSRC, "fa_calls.cpp"), "-o", tmp,
           "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        why = "" if r.returncode == 0 else f"{r.stdout}\n{r.stderr}"
    except OSError as e:
        why = str(e)
    if why:
        sys.stderr.write(f"the module _calls was not built (the library works without it, short calls take longer): "
                         f"g++ failed on fa_calls.cpp:\n{why}\n")
        return None
    os.replace(tmp, CALLS)
    return CALLS


def build(ptxas_verbose: bool = False, quiet: bool = True) -> str:
    """Compile every CUDA source and link the library; returns its path."""
    nvcc = nvcc_path()
    os.makedirs(OBJ, exist_ok=True)
    srcs = sources()
    logs = []
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        calls = ex.submit(build_calls)
        futs = [ex.submit(_compile, nvcc, s, ptxas_verbose) for s in srcs]
        objs = []
        for f in futs:
            obj, log = f.result()
            objs.append(obj)
            logs.append(log)
        calls.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if not quiet or ptxas_verbose:
        sys.stdout.write("".join(logs))
    return LIB


if __name__ == "__main__":
    print(build(ptxas_verbose="--ptxas-verbose" in sys.argv, quiet=False))
