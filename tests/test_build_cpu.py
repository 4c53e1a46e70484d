"""The build step on machines other than the one it was written on: nothing is compiled
here, the commands and the files that they leave are looked at."""
import os
import subprocess
import sys
import sysconfig

import pytest

from rope_frequency_sparse_b200 import atf, build


@pytest.fixture
def fake(monkeypatch, tmp_path):
    """A build into an empty folder whose compilers write their output file and do nothing else."""
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libatf.so"))
    monkeypatch.setattr(build, "HERE", str(tmp_path))
    commands = []

    def run(cmd, **kw):
        commands.append(cmd)
        if cmd[0] == "g++" and fake_gxx["fails"]:
            return subprocess.CompletedProcess(cmd, 1, "", "Python.h: No such file or directory")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    fake_gxx = {"fails": False}
    monkeypatch.setattr(build.subprocess, "run", run)
    return commands, fake_gxx


def _modules():
    return sorted(f for f in os.listdir(build.HERE) if f.startswith("_tensor_calls"))


def test_the_library_is_built_without_torch(fake, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not _modules() and "torch" in capsys.readouterr().err


def test_the_library_is_linked_where_its_torch_module_fails(fake):
    fake[1]["fails"] = True
    with pytest.raises(RuntimeError, match="Python.h"):
        build.build()
    assert os.path.exists(build.LIB)


@pytest.mark.parametrize("how", ["path", "name", "link"])
def test_cuda_headers_are_found_however_nvcc_is_named(fake, monkeypatch, tmp_path, how):
    home = tmp_path / "cuda"
    for f in (home / "bin" / "nvcc", home / "include" / "cuda_runtime_api.h"):
        f.parent.mkdir(parents=True)
        f.write_text("#!/bin/sh\n")
    nvcc = home / "bin" / "nvcc"
    nvcc.chmod(0o755)
    if how == "link":
        (tmp_path / "elsewhere").mkdir()
        (tmp_path / "elsewhere" / "nvcc").symlink_to(nvcc)
    monkeypatch.setenv("PATH", str(home / "bin") + os.pathsep + os.environ["PATH"])
    monkeypatch.setattr(build, "NVCC", {"path": str(nvcc), "name": "nvcc", "link": str(tmp_path / "elsewhere" / "nvcc")}[how])
    build.build()
    (gxx,) = [c for c in fake[0] if c[0] == "g++"]
    assert str((home / "include").resolve()) in [os.path.realpath(a[2:]) for a in gxx if a.startswith("-I")]


def test_another_torch_or_python_gets_a_module_of_its_own(fake, monkeypatch):
    import torch

    build.build()
    build.build()
    assert len(_modules()) == 1 and len([c for c in fake[0] if c[0] == "g++"]) == 1
    monkeypatch.setattr(torch, "__version__", "99.1.2")
    build.build()
    assert len(_modules()) == 2 and any("99.1.2" in f for f in _modules())
    suffix = sysconfig.get_config_var
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda n: ".cpython-399.so" if n == "EXT_SUFFIX" else suffix(n))
    build.build()
    assert len(_modules()) == 3


def test_a_module_of_another_torch_is_not_loaded(monkeypatch):
    import torch

    build.build()
    monkeypatch.setattr(atf, "_calls", None)
    monkeypatch.setattr(torch, "__version__", "99.1.2")
    with pytest.raises(RuntimeError, match="99.1.2.*is not built"):
        atf._tensor_calls()
