"""When the build compiles the binding of the prompt-side calls again (no compiler runs here: commands are recorded)."""
import os
import shutil
import subprocess

import pytest
import torch

from group_wise_weight_b200 import build as wqbuild


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """An up-to-date build whose binding lies under tmp_path; what build() runs from here on."""
    wqbuild.build()
    binding = tmp_path / "_wq_torch.so"
    shutil.copy2(wqbuild.BINDING, binding)
    monkeypatch.setattr(wqbuild, "BINDING", str(binding))
    if hasattr(wqbuild, "BINDING_STAMP"):
        stamp = tmp_path / "stamp"
        shutil.copy2(wqbuild.BINDING_STAMP, stamp)
        monkeypatch.setattr(wqbuild, "BINDING_STAMP", str(stamp))
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(wqbuild.subprocess, "run", run)
    return ran


def test_nothing_is_compiled_when_nothing_changed(commands):
    assert wqbuild.build() == wqbuild.LIB and commands == []


def test_another_torch_compiles_the_binding_again(commands, monkeypatch):
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    wqbuild.build()
    assert [c[0] for c in commands] == ["g++"]
    wqbuild.build()
    assert len(commands) == 1


def test_another_python_compiles_the_binding_again(commands, monkeypatch):
    known = wqbuild.sysconfig.get_config_var
    monkeypatch.setattr(wqbuild.sysconfig, "get_config_var", lambda n: "cpython-399" if n == "SOABI" else known(n))
    wqbuild.build()
    assert [c[0] for c in commands] == ["g++"]


def test_a_newer_source_compiles_the_binding_again(commands):
    os.utime(wqbuild.BINDING, (0, 0))
    wqbuild.build()
    assert [c[0] for c in commands] == ["g++"]


def test_without_headers_the_library_is_built_all_the_same(commands, monkeypatch, tmp_path):
    """libwq.so serves the calls that do not go through the binding; those that do say what is missing."""
    os.utime(wqbuild.BINDING, (0, 0))
    paths = wqbuild.sysconfig.get_paths()
    monkeypatch.setattr(wqbuild.sysconfig, "get_paths", lambda: {**paths, "include": str(tmp_path)})
    with pytest.warns(UserWarning, match="Python.h"):
        assert wqbuild.build() == wqbuild.LIB
    assert commands == [] and not os.path.exists(wqbuild.BINDING)
    import group_wise_weight_b200 as wq
    monkeypatch.setattr(wq, "_native_module", None)
    monkeypatch.setattr(wq, "BINDING_PATH", wqbuild.BINDING)
    wq.lib()
    with pytest.raises(RuntimeError, match="_wq_torch.so not found"):
        wq.wq_quantize_int8_tokens(torch.zeros(4, 256))


def test_without_a_compiler_the_library_is_built_all_the_same(commands, monkeypatch):
    os.utime(wqbuild.BINDING, (0, 0))
    known = shutil.which
    monkeypatch.setattr(wqbuild.shutil, "which", lambda n: None if n == "g++" else known(n))
    with pytest.warns(UserWarning, match="g\\+\\+ not found"):
        assert wqbuild.build() == wqbuild.LIB
    assert commands == []


def test_a_binding_that_does_not_compile_fails_the_build(commands, monkeypatch):
    os.utime(wqbuild.BINDING, (0, 0))
    monkeypatch.setattr(wqbuild.subprocess, "run", lambda cmd, **kw: subprocess.CompletedProcess(cmd, 1, "", "error: x"))
    with pytest.raises(RuntimeError, match="error: x"):
        wqbuild.build()
