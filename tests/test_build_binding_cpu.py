"""Host-side checks of what the build needs: the C library hipcc alone, the
binding's _tensors.so also torch, g++ and Python's headers."""
import os
import shutil
import subprocess

import pytest

from state_space_sequence_exp_amd import build as b


@pytest.fixture
def compilers(monkeypatch, tmp_path):
    """Compilers that write empty files, into a folder of their own; the commands run."""
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(b.subprocess, "run", run)
    lib = str(tmp_path / "libm3ssm.so")
    monkeypatch.setattr(b, "LIB_PATH", lib)
    monkeypatch.setattr(b, "TENSORS_PATH", str(tmp_path / "_tensors.so"))
    which = shutil.which
    monkeypatch.setattr(b.shutil, "which", lambda name: name if name in ("hipcc", "g++") else which(name))
    monkeypatch.setattr(b, "_hipcc", lambda: "hipcc")
    return ran, lib


def ran_gxx(ran):
    return any(cmd[0] == "g++" for cmd in ran)


def test_both_are_built(compilers):
    ran, lib = compilers
    assert b.build(out=lib) == lib and ran_gxx(ran)
    assert os.path.exists(lib) and os.path.exists(b.TENSORS_PATH)


def test_library_alone(compilers):
    ran, lib = compilers
    assert b.build(out=lib, binding=False) == lib and not ran_gxx(ran)
    assert os.path.exists(lib) and not os.path.exists(b.TENSORS_PATH)


def test_library_without_torch(compilers, monkeypatch, capfd):
    ran, lib = compilers
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: None)
    assert b.build(out=lib) == lib and not ran_gxx(ran) and os.path.exists(lib)
    assert "torch is not installed" in capfd.readouterr().err


def test_without_a_compiler_says_so(compilers, monkeypatch):
    ran, lib = compilers
    monkeypatch.setattr(b.shutil, "which", lambda name: None)
    with pytest.raises(RuntimeError, match="--library-only"):
        b.build(out=lib)
    assert os.path.exists(lib)


def test_tensors_compile_without_warnings(monkeypatch, tmp_path, capfd):
    monkeypatch.setattr(b, "TENSORS_PATH", str(tmp_path / "_tensors.so"))
    b.build_tensors(verbose=True)
    assert "warning" not in capfd.readouterr().err
