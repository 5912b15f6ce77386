"""Build libqidit.so (the C-ABI library) in-tree with nvcc for sm_103a.

    python -m diffusion_transformer_text_gb300.build [--force]

Translation units compile in parallel; the output goes to
diffusion_transformer_text_gb300/_build/libqidit.so (git-ignored). Beside it goes qi_tensors.so, the
part of the Python binding that is compiled against PyTorch's headers.
"""
from __future__ import annotations

import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libqidit.so")
TENSORS = os.path.join(BUILD, "qi_tensors.so")  # the binding's reader of tensor arguments (csrc/tensors.cpp)
SOURCES = ["qidit.cu", "gemm.cu", "attention.cu", "kernels_small.cu", "gemm_noalloc.cu", "prefix_attention.cu",
           "prefix_attention_few.cu", "paged_attention.cu", "batch_ops.cu", "rope_ops.cu"]
HEADERS = ["ptx.cuh", "internal.h", "prefix_attention.cuh", "values.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
         "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libqidit.so")


def _torch_dir() -> str | None:
    import importlib.util
    spec = importlib.util.find_spec("torch")
    return list(spec.submodule_search_locations)[0] if spec is not None and spec.submodule_search_locations else None


def _torch_version() -> str:
    if _torch_dir() is None:
        return ""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return f.read()


def _build_tensors() -> None:
    """qi_tensors.so, a CPython module over PyTorch's headers (host code only); without PyTorch there is none, and
    the library alone is built."""
    t, py = _torch_dir(), sysconfig.get_paths()["include"]
    if t is None:
        return
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = TENSORS + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-I" + py, "-I" + os.path.join(t, "include"),
           "-I" + os.path.join(t, "include", "torch", "csrc", "api", "include"), "-I" + os.path.join(cuda, "include"),
           os.path.join(CSRC, "tensors.cpp"), "-o", tmp, "-L" + os.path.join(t, "lib"), "-ltorch_python", "-ltorch_cpu",
           "-lc10", "-Wl,-rpath," + os.path.join(t, "lib")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on tensors.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, TENSORS)


def _fingerprint() -> str:
    h = hashlib.sha256()
    for name in SOURCES + HEADERS + ["tensors.cpp"]:
        with open(os.path.join(CSRC, name), "rb") as f:
            h.update(name.encode() + f.read())
    with open(os.path.join(ROOT, "include", "qidit.h"), "rb") as f:
        h.update(f.read())
    h.update(" ".join(ARCH + FLAGS).encode())
    h.update(os.uname().machine.encode())
    h.update(sys.version.encode() + _torch_version().encode())
    return h.hexdigest()


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if sources changed) and return the path of libqidit.so."""
    os.makedirs(BUILD, exist_ok=True)
    stamp = os.path.join(BUILD, "libqidit.stamp")
    fp = _fingerprint()
    if not force and os.path.exists(LIB) and os.path.exists(stamp) and (os.path.exists(TENSORS) or _torch_dir() is None):
        with open(stamp) as f:
            if f.read().strip() == fp:
                return LIB
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        tensors = ex.submit(_build_tensors)
        results = list(ex.map(compile_one, SOURCES))
        tensors.result()
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    with open(stamp, "w") as f:
        f.write(fp)
    with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
        for o, log in results:
            f.write(f"== {os.path.basename(o)}\n{log}\n")
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
