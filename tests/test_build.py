"""What build() makes, of what, and when: the CUDA library by nvcc alone, the compiled reader of tensors beside it."""
import ctypes
import importlib
import os
import stat
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture()
def b(monkeypatch, tmp_path):
    """build.py on a library of one small function, in folders of its own."""
    b = importlib.import_module("diffusion_transformer_text_gb300.build")
    out, src = tmp_path / "_build", tmp_path / "csrc"
    src.mkdir()
    (src / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    (src / "tensors.cpp").write_text('extern "C" int two() { return 2; }\n')
    for name, value in dict(CSRC=src, BUILD=out, LIB=out / "libqidit.so", TENSORS=out / "qi_tensors.so").items():
        monkeypatch.setattr(b, name, str(value))
    monkeypatch.setattr(b, "SOURCES", ["one.cu"])
    monkeypatch.setattr(b, "HEADERS", [])
    monkeypatch.setattr(b, "_torch_dir", lambda: str(tmp_path / "torch"))
    monkeypatch.setattr(b, "_torch_version", lambda: "1")
    return b


def _compiler(monkeypatch, tmp_path, status=0):
    """A CXX that says that it ran, and writes its output unless it fails; (a function that counts its runs)."""
    log, path = tmp_path / "runs", tmp_path / f"cxx{status}"
    path.write_text(f"#!/bin/sh\necho run >> {log}\n" + (f"echo no headers >&2\nexit {status}\n" if status else
                    'while [ "$1" != -o ]; do shift; done\necho module > "$2"\n'))
    path.chmod(path.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("CXX", str(path))
    return lambda: len(log.read_text().split()) if log.exists() else 0


@pytest.mark.parametrize("cxx", ["fails", "absent", "/bin/true"])
def test_without_the_reader_the_library_is_built(b, monkeypatch, tmp_path, cxx):
    if cxx == "fails":
        _compiler(monkeypatch, tmp_path, 1)
    else:
        monkeypatch.setenv("CXX", cxx if cxx[0] == "/" else str(tmp_path / "absent"))
    with pytest.warns(RuntimeWarning, match="qi_tensors.so was not built"):
        assert b.build() == b.LIB
    assert ctypes.CDLL(b.LIB).one() == 1
    assert not os.path.exists(b.TENSORS) and b.tensors_failure()
    assert cxx != "fails" or "no headers" in b.tensors_failure()
    # ... and the next build has only the reader to make
    runs = _compiler(monkeypatch, tmp_path)
    before = os.stat(b.LIB).st_mtime_ns
    monkeypatch.setattr(b, "nvcc", lambda: pytest.fail("CUDA files compiled again"))
    had = runs()
    b.build()
    assert runs() == had + 1 and os.path.exists(b.TENSORS) and b.tensors_failure() == ""
    assert os.stat(b.LIB).st_mtime_ns == before


def test_what_is_compiled_again(b, monkeypatch, tmp_path):
    runs = _compiler(monkeypatch, tmp_path)
    b.build()
    b.build()
    assert runs() == 1
    # another PyTorch, Python or compiler: the reader alone, and no nvcc is asked for
    nvcc = b.nvcc
    monkeypatch.setattr(b, "nvcc", lambda: pytest.fail("CUDA files compiled again"))
    monkeypatch.setattr(b, "_torch_version", lambda: "2")
    b.build()
    assert runs() == 2
    monkeypatch.setattr(sys, "version", sys.version + " another")
    b.build()
    assert runs() == 3
    monkeypatch.setenv("CXX", os.environ["CXX"] + " -g")
    b.build()
    assert runs() == 4
    # an interpreter without PyTorch uses the library as it is, and leaves the reader to the others
    monkeypatch.setattr(b, "_torch_dir", lambda: None)
    b.build()
    assert runs() == 4 and os.path.exists(b.TENSORS)
    monkeypatch.setattr(b, "_torch_dir", lambda: str(tmp_path / "torch"))
    b.build()
    assert runs() == 4
    # another CUDA file: the library alone
    monkeypatch.setattr(b, "nvcc", nvcc)
    with open(os.path.join(b.CSRC, "one.cu"), "w") as f:
        f.write('extern "C" int one() { return 11; }\n')
    before = os.stat(b.LIB).st_mtime_ns
    b.build()
    assert runs() == 4 and os.stat(b.LIB).st_mtime_ns != before
    # a reader that can't be made again does not stay as that of another PyTorch
    _compiler(monkeypatch, tmp_path, 1)
    with pytest.warns(RuntimeWarning):
        b.build()
    assert not os.path.exists(b.TENSORS) and ctypes.CDLL(b.LIB).one() == 11


def test_the_first_call_that_needs_the_reader_says_why_there_is_none(tmp_path):
    importlib.import_module("diffusion_transformer_text_gb300").build()
    code = f"""
import diffusion_transformer_text_gb300 as q
import sys
b = sys.modules["diffusion_transformer_text_gb300.build"]
q.TENSORS = b.TENSORS = {str(tmp_path / "qi_tensors.so")!r}
open(b.TENSORS + ".log", "w").write("no headers here")
q.lib()
for _ in range(2):
    try:
        q._describe(None)
    except RuntimeError as e:
        assert "no headers here" in str(e) and "build()" in str(e), e
    else:
        raise SystemExit("no error")
"""
    subprocess.run([sys.executable, "-c", code], check=True, cwd=ROOT)
