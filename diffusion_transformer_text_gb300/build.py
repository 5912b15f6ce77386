"""Build libqidit.so (the C-ABI library) in-tree with nvcc for sm_103a.

    python -m diffusion_transformer_text_gb300.build [--force]

Translation units compile in parallel; the output goes to
diffusion_transformer_text_gb300/_build/libqidit.so (git-ignored). Beside it goes qi_tensors.so, the
part of the Python binding that is compiled against PyTorch's headers.
"""
from __future__ import annotations

import hashlib
import os
import shlex
import shutil
import subprocess
import sys
import sysconfig
import warnings
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
    return "" if _torch_dir() is None else _read(os.path.join(_torch_dir(), "version.py"))


def _tensors_command() -> list:
    """How qi_tensors.so is compiled (host code over Python's and PyTorch's headers), but for its output."""
    t, py = _torch_dir(), sysconfig.get_paths()["include"]
    return [*shlex.split(os.environ.get("CXX", "g++")), "-O2", "-std=c++17", "-shared", "-fPIC", "-I" + py, "-I" + os.path.join(t, "include"),
            "-I" + os.path.join(t, "include", "torch", "csrc", "api", "include"), os.path.join(CSRC, "tensors.cpp"),
            "-L" + os.path.join(t, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-Wl,-rpath," + os.path.join(t, "lib")]


def _remove(path: str) -> None:
    if os.path.exists(path):
        os.remove(path)


def _build_tensors(force: bool = False) -> str:
    """qi_tensors.so, a CPython module; without PyTorch there is none. Returns why it could not be made, or "". Only
    the calls that read their tensors by it need it, so what went wrong is kept (tensors_failure) for the first of them."""
    if _torch_dir() is None:
        return ""
    stamp, log, cmd = TENSORS + ".stamp", TENSORS + ".log", _tensors_command()
    h = hashlib.sha256()
    with open(os.path.join(CSRC, "tensors.cpp"), "rb") as f:
        h.update(f.read())
    h.update("\0".join([*cmd, os.uname().machine, sys.version, _torch_version()]).encode())
    if not force and os.path.exists(TENSORS) and _read(stamp) == h.hexdigest():
        return ""
    tmp, why = TENSORS + ".tmp", ""
    _remove(tmp)
    try:
        r = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
        if r.returncode != 0 or not os.path.exists(tmp):
            why = f"{cmd[0]} failed on tensors.cpp (status {r.returncode}):\n{r.stdout}\n{r.stderr}"
    except OSError as e:
        why = f"{cmd[0]} could not be run: {e}"
    _remove(stamp)
    if why:  # (an older module may be of another PyTorch)
        _remove(TENSORS)
        with open(log, "w") as f:
            f.write(why)
        return why
    os.replace(tmp, TENSORS)
    _remove(log)
    with open(stamp, "w") as f:
        f.write(h.hexdigest())
    return ""


def tensors_failure() -> str:
    """Why the last build made no qi_tensors.so, "" if it did."""
    return _read(TENSORS + ".log")


def _read(path: str) -> str:
    """A text file's contents, "" if there is none."""
    if not os.path.exists(path):
        return ""
    with open(path) as f:
        return f.read().strip()


def _fingerprint() -> str:
    h = hashlib.sha256()
    for name in SOURCES + HEADERS:
        with open(os.path.join(CSRC, name), "rb") as f:
            h.update(name.encode() + f.read())
    with open(os.path.join(ROOT, "include", "qidit.h"), "rb") as f:
        h.update(f.read())
    h.update(" ".join(ARCH + FLAGS).encode())
    h.update(os.uname().machine.encode())
    return h.hexdigest()


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if sources changed) and return the path of libqidit.so. The binding's qi_tensors.so is compiled
    beside it; if that fails the library is there all the same, and a warning says why."""
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(1) as ex:
        tensors = ex.submit(_build_tensors, force)
        _build_library(force, verbose)
        why = tensors.result()
    if why:
        warnings.warn(f"qi_tensors.so was not built, so qk_norm_rope and paged_attention will raise: {why}", RuntimeWarning,
                      stacklevel=2)
    return LIB


def _build_library(force: bool, verbose: bool) -> None:
    stamp = os.path.join(BUILD, "libqidit.stamp")
    fp = _fingerprint()
    if not force and os.path.exists(LIB) and _read(stamp) == fp:
        return
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with ThreadPoolExecutor(len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
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


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
