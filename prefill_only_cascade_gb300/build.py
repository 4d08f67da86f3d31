"""Build libquail.so in-tree for sm_103a (GB300) with nvcc.

Each translation unit in csrc/ is compiled in parallel to an object under _build/, then
linked into prefill_only_cascade_gb300/libquail.so (CUDA runtime linked statically). Beside them the
host side of the binding's paged calls, _paged_calls.so, which needs PyTorch's and Python's headers; the
binding does without it where they are missing.
Run: python prefill_only_cascade_gb300/build.py
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libquail.so")
CALLS = os.path.join(PKG, "_paged_calls.so")
SOURCES = ["api.cu", "api_paged.cu", "cascade.cu", "evict.cu", "head.cu", "kv_plan.cu",
           "noalloc.cu", "paged.cu", "paged_rows.cu", "fp4_decode.cu", "prefill.cu", "quantize.cu", "scores.cu", "select.cu",
           "shard.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags(extra=()):
    return ["-O3", "-std=c++17", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC",
            "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, *extra]


def _torch_home() -> str:
    """Where PyTorch is installed, found without loading it."""
    import importlib.util

    try:
        spec = importlib.util.find_spec("torch")
    except ValueError as e:  # a stand-in among the loaded modules
        raise ImportError(str(e)) from e
    if spec is None or spec.origin is None:
        raise ImportError("PyTorch is not installed")
    return os.path.dirname(spec.origin)


def build_calls(nvcc: str) -> str | None:
    """_paged_calls.so; None (and why, on stderr) where it cannot be built."""
    import sysconfig

    tmp = CALLS + ".tmp"
    try:
        home = _torch_home()
        includes = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
                    sysconfig.get_paths()["include"],
                    os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include"),
                    os.path.join(ROOT, "include")]
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", *["-I" + x for x in includes],
               os.path.join(CSRC, "paged_calls.cpp"), "-o", tmp, "-L" + os.path.join(home, "lib"),
               "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        log = r.stderr if r.returncode != 0 else ""
    except (ImportError, OSError) as e:
        log = str(e)
    if log:
        print(f"_paged_calls.so not built, the binding checks arguments in Python:\n{log[-2000:]}", file=sys.stderr)
        if os.path.exists(CALLS):
            os.remove(CALLS)
        return None
    os.replace(tmp, CALLS)
    return CALLS


def build(verbose: bool = False, ptxas_verbose: bool = False) -> str:
    nvcc = nvcc_path()
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc, *_flags(extra), "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = ex.submit(build_calls, nvcc)
        results = list(ex.map(compile_one, SOURCES))
        calls.result()
    if verbose or ptxas_verbose:
        for _, log in results:
            if log.strip():
                print(log)
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, ptxas_verbose="-v" in sys.argv))
