"""The library of the C ABI is built with hipcc alone; the torch-facing marshalling is an addition that a
machine without torch, its HIP headers, Python's headers or a C++ compiler does without (no GPU, nothing
compiled here)."""
import os
import shutil
import subprocess
import sys

import pytest

from w4a4_post_quantized_zigzag_amd import binding
from w4a4_post_quantized_zigzag_amd import build as b


@pytest.fixture
def bare(tmp_path, monkeypatch):
    """build() with its outputs in a folder of its own and the compilers replaced: hipcc succeeds and writes
    its -o, anything else counts as the C++ compiler and is recorded."""
    pkg = tmp_path / "pkg"
    pkg.mkdir()
    monkeypatch.setattr(b, "PKG", str(pkg))
    monkeypatch.setattr(b, "BUILD", str(pkg / "_build"))
    monkeypatch.setattr(b, "LIB", str(pkg / "libw4a4.so"))
    calls = []

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        if cmd[0] != b.HIPCC:
            calls.append(cmd)
            if run.cxx_fails:
                return subprocess.CompletedProcess(cmd, 1, "", "some error")
        with open(out, "w") as f:
            f.write(cmd[0])
        return subprocess.CompletedProcess(cmd, 0, "", "")

    run.cxx_fails, run.calls = False, calls
    monkeypatch.setattr(b.subprocess, "run", run)
    (pkg / "_decode.so").write_text("of an older library")
    return pkg, run


def test_without_torch(bare, monkeypatch, capsys):
    pkg, run = bare
    monkeypatch.setitem(sys.modules, "torch", None)
    monkeypatch.setitem(sys.modules, "torch.utils.cpp_extension", None)
    assert b.build() == str(pkg / "libw4a4.so")
    assert (pkg / "libw4a4.so").exists() and not run.calls
    # a module linked against an older library does not stay beside the new one
    assert not (pkg / "_decode.so").exists()
    assert "torch" in capsys.readouterr().out


def test_without_a_compiler(bare, monkeypatch, capsys):
    pkg, run = bare
    monkeypatch.setenv("CXX", "no-such-compiler")
    assert b.build() == str(pkg / "libw4a4.so")
    assert not run.calls and not (pkg / "_decode.so").exists()
    assert "no-such-compiler" in capsys.readouterr().out


def test_without_python_headers(bare, monkeypatch, tmp_path, capsys):
    pkg, run = bare
    monkeypatch.setattr(b.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert b.build() == str(pkg / "libw4a4.so")
    assert not run.calls and not (pkg / "_decode.so").exists()
    assert "Python.h" in capsys.readouterr().out


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a compiler to be found")
def test_a_failing_compile_is_an_error(bare):
    pkg, run = bare
    run.cxx_fails = True
    with pytest.raises(RuntimeError, match="some error"):
        b.build()
    assert (pkg / "libw4a4.so").exists() and not (pkg / "_decode.so").exists()


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a compiler to be found")
def test_both_parts(bare, capsys):
    pkg, run = bare
    assert b.build() == str(pkg / "libw4a4.so")
    assert len(run.calls) == 1 and (pkg / "_decode.so").read_text() == run.calls[0][0]
    assert "_decode.so" in capsys.readouterr().out


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a compiler to be found")
def test_hipcc_by_name(bare, monkeypatch):
    """HIPCC may be a bare name; HIP's headers are still found."""
    pkg, run = bare
    monkeypatch.setattr(b, "HIPCC", "hipcc")
    b.build()
    dirs = [d for f, d in zip(run.calls[0], run.calls[0][1:]) if f == "-isystem"]
    assert any(os.path.exists(os.path.join(d, "hip", "hip_runtime.h")) and os.path.isabs(d) for d in dirs)


def test_calls_without_the_module_raise(monkeypatch, tmp_path):
    """No fallback: without the module the single-token calls say how to build it."""
    import torch
    monkeypatch.setattr(binding, "_native", None)
    monkeypatch.setitem(sys.modules, binding.__package__ + "._decode", None)
    with pytest.raises(RuntimeError, match="build"):
        binding.gemv_w4g(torch.zeros(1, 32), None, None)
    assert os.path.exists(binding.LIB_PATH)
