"""The build without the operators' Python module: the library is linked all the same."""
from __future__ import annotations

import subprocess

import pytest

from bit_routed_expert_amd import build as B


@pytest.fixture
def dry(monkeypatch, tmp_path):
    """build() in a folder of its own, its compilers replaced by stubs; returns the link's output path."""
    lib, binding = tmp_path / "libstrata_moe.so", tmp_path / "_binding.so"
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(B, "LIB", str(lib))
    monkeypatch.setattr(B, "BINDING", str(binding))
    monkeypatch.setattr(B, "_compile", lambda src: src + ".o")
    monkeypatch.setattr(B, "_compile_host", lambda ns: ns + ".o")
    monkeypatch.setattr(B, "_compile_host_common", lambda: "host.o")

    def run(cmd, **kw):
        failed = "-shared" in cmd and any(str(c).endswith("binding.cpp") for c in cmd)
        if not failed:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, int(failed), "", "Python.h: No such file or directory")
    monkeypatch.setattr(B.subprocess, "run", run)
    return lib, binding


def test_the_library_is_built_where_the_binding_is_not(dry):
    lib, binding = dry
    binding.write_text("of an earlier build")
    with pytest.warns(RuntimeWarning, match="Python.h"):
        assert B.build() == str(lib)
    assert lib.exists() and not binding.exists()


def test_a_library_that_does_not_compile_still_raises(dry, monkeypatch):
    lib, _ = dry

    def broken(src):
        raise RuntimeError(f"hipcc failed for {src}")
    monkeypatch.setattr(B, "_compile", broken)
    with pytest.raises(RuntimeError, match="hipcc failed"):
        B.build()
    assert not lib.exists()
