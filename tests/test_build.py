"""Steps of the build, on the host."""
import os
import subprocess

import pytest

from block_scaled_fp4_histogram_amd import build as B


def test_library_is_built_without_the_host_compiler(tmp_path, monkeypatch):
    """The C ABI and the layer need hipcc only; the torch binding is a step of its own, whose failure is an
    error and leaves the library in place."""
    ran = []

    def fake(cmd, **kw):
        ran.append(cmd[0])
        if cmd[0] != B.HIPCC:
            return subprocess.CompletedProcess(cmd, 1, "", "no such compiler")
        open(cmd[-1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(B, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(B, "BINDING", str(tmp_path / "binding.so"))
    monkeypatch.setattr(B.subprocess, "run", fake)
    monkeypatch.setenv("CXX", "a-compiler-that-is-not-there")
    assert B.build() == str(tmp_path / "lib.so") and ran == [B.HIPCC]
    with pytest.raises(RuntimeError, match="no such compiler"):
        B.build_binding()
    assert os.listdir(tmp_path) == ["lib.so"]


def test_missing_host_compiler_is_named(tmp_path, monkeypatch):
    monkeypatch.setattr(B, "BINDING", str(tmp_path / "binding.so"))
    monkeypatch.setenv("CXX", str(tmp_path / "none"))
    with pytest.raises(RuntimeError, match="none"):
        B.build_binding()
