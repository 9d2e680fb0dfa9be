"""Build libbiv.so in-tree with nvcc for sm_103a (GB300).

One translation unit per kernel family, compiled in parallel, then linked
into ``invariant_verify_gb300/libbiv.so`` (git-ignored).  The CUDA runtime
is linked statically, so the library only needs the driver at run time.
Beside it ``_biv_torch.so``, the Python binding of the small calls.
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

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libbiv.so")
TORCH_LIB = os.path.join(HERE, "_biv_torch.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

SOURCES = ["biv_api.cu", "biv_gemm.cu", "biv_select.cu", "biv_attn.cu", "biv_rowops.cu", "biv_draft.cu",
           "biv_paged.cu", "biv_sample.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I", INCLUDE]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: libbiv needs the CUDA toolkit to build")
    return cand


def _stale(obj: str, deps: list) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, verbose_ptxas: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    # every header of the library: an object is rebuilt when any of them changes
    headers = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h")))
    deps = [os.path.join(CSRC, src), *headers, os.path.join(INCLUDE, "biv.h")]
    if _stale(obj, deps) or verbose_ptxas:
        cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose_ptxas:
            cmd += ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose_ptxas:
            sys.stderr.write(r.stderr)
    return obj


def _compile_torch() -> None:
    """The binding of the small calls (csrc/biv_torch.cpp), for the torch and the
    Python that run this.  A file beside it holds the command that made it, with
    torch's version: another one rebuilds it, whatever the files' times say.  The
    library itself needs no torch: without one there is nothing to bind."""
    torch = importlib.util.find_spec("torch")
    if torch is None:
        return
    torch_dir = torch.submodule_search_locations[0]
    src = os.path.join(CSRC, "biv_torch.cpp")
    with open(os.path.join(torch_dir, "version.py")) as f:
        version = re.search(r"__version__ = ['\"]([^'\"]+)['\"]", f.read()).group(1)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [INCLUDE, os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", f'-DBIV_TORCH_VERSION="{version}"', *(f"-I{d}" for d in inc),
           src, "-o", TORCH_LIB + ".tmp", "-L" + os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-lc10_cuda"]
    made = "\n".join([*cmd, sysconfig.get_config_var("SOABI") or ""])
    if not _stale(TORCH_LIB, [src, os.path.join(INCLUDE, "biv.h")]) and os.path.exists(TORCH_LIB + ".cmd"):
        with open(TORCH_LIB + ".cmd") as f:
            if f.read() == made:
                return
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on biv_torch.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(TORCH_LIB + ".tmp", TORCH_LIB)
    with open(TORCH_LIB + ".cmd", "w") as f:
        f.write(made)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    if force:
        for f in os.listdir(BUILD):
            os.remove(os.path.join(BUILD, f))
    if force and os.path.exists(TORCH_LIB):
        os.remove(TORCH_LIB)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_torch)
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas), SOURCES))
        binding.result()
    if force or _stale(LIB, objs):
        cmd = [nvcc(), *ARCH, "-shared", "-o", LIB + ".tmp", *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
