"""The build step on machines other than the one it was written on: nothing is compiled
here, the commands and the files that they leave are looked at."""
import os
import subprocess
import sys

import pytest

from rope_frequency_sparse_b200 import build


@pytest.fixture
def fake(monkeypatch, tmp_path):
    """A build into an empty folder whose compilers write their output file and do nothing else."""
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libatf.so"))
    monkeypatch.setattr(build, "TENSOR_CALLS", str(tmp_path / "_tensor_calls.so"))
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


def test_the_library_is_built_without_torch(fake, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.TENSOR_CALLS) and "torch" in capsys.readouterr().err


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
