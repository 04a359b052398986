"""What build() needs: hipcc for the library, torch and a host compiler for the
Python module alone.  No compiler runs here."""
import importlib.util
from types import SimpleNamespace

import pytest

from bit_block_quantized_nvfp4_amd import build as b


@pytest.fixture
def steps(monkeypatch, tmp_path):
    """Commands run, with files put in the places they would write."""
    run = []

    class Popen:
        returncode = 0

        def __init__(self, cmd, **kw):
            run.append(cmd)
            open(cmd[cmd.index("-o") + 1], "w").close()

        def communicate(self):
            return b"", None

    def call(cmd, **kw):
        Popen(cmd)
        return SimpleNamespace(returncode=0, stdout=b"")

    monkeypatch.setattr(b, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(b, "hipcc", lambda: "/opt/rocm/bin/hipcc")
    monkeypatch.setattr(b.subprocess, "Popen", Popen)
    monkeypatch.setattr(b.subprocess, "run", call)
    return SimpleNamespace(run=run, lib=tmp_path / "lib.so", module=tmp_path / "_binding.so")


def test_both_are_built(steps):
    assert b.build() == str(steps.lib) and steps.lib.exists() and steps.module.exists()


def test_the_library_needs_no_torch(steps, monkeypatch):
    real = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else real(name, *a))
    monkeypatch.setitem(__import__("sys").modules, "torch", None)  # importing it fails
    assert b.build() == str(steps.lib)
    assert steps.lib.exists() and not steps.module.exists()
    assert not any("binding.cpp" in str(c) for c in steps.run)


def test_the_library_is_in_place_when_the_module_fails(steps, monkeypatch):
    def fails(out):
        raise RuntimeError("no headers")

    monkeypatch.setattr(b, "binding_command", fails)
    with pytest.raises(RuntimeError, match="no headers"):
        b.build()
    assert steps.lib.exists()


def test_the_module_takes_another_compiler_where_there_is_no_gxx(monkeypatch):
    monkeypatch.delenv("CXX", raising=False)
    monkeypatch.setattr(b.shutil, "which", lambda c: None if c == "g++" else c)
    assert b.cxx().endswith("amdclang++")
    monkeypatch.setattr(b.shutil, "which", lambda c: None)
    with pytest.raises(RuntimeError, match="library itself is built"):
        b.cxx()
