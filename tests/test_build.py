"""What the build makes where a part of the toolchain is missing, with a stand-in for nvcc."""
import importlib.util
import os
import stat
import sys

import pytest
import torch

from conftest import ROOT

BUILD = os.path.join(ROOT, "sequence_blockwise_softmax_gb300", "build.py")


def script(path, text):
    path.write_text("#!/bin/sh\n" + text)
    path.chmod(path.stat().st_mode | stat.S_IXUSR)
    return str(path)


@pytest.fixture
def build(tmp_path, monkeypatch):
    """build.py writing to a folder of its own; its nvcc creates whatever -o names and logs that."""
    spec = importlib.util.spec_from_file_location("build_under_test", BUILD)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    for name in ("LIB", "BINDING"):
        if hasattr(module, name):
            monkeypatch.setattr(module, name, str(tmp_path / "_lib" / os.path.basename(getattr(module, name))))
    monkeypatch.setattr(module, "OUT_DIR", str(tmp_path / "_lib"))
    module.log = tmp_path / "nvcc.log"
    module.log.write_text("")
    monkeypatch.setenv("NVCC", script(tmp_path / "nvcc", """
while [ $# -gt 1 ]; do
  if [ "$1" = -o ]; then : > "$2"; echo "$2" >> "%s"; fi
  shift
done
""" % module.log))
    return module


def without_gxx(tmp_path, monkeypatch):
    bin_dir = tmp_path / "bin"
    bin_dir.mkdir()
    script(bin_dir / "g++", "echo no such header >&2; exit 1\n")
    monkeypatch.setenv("PATH", str(bin_dir) + os.pathsep + os.environ["PATH"])


def test_the_library_does_not_need_the_binding(build, tmp_path, monkeypatch):
    """A C caller's machine: no compiler or headers for the torch binding.  The library is there all
    the same, and the failure is reported."""
    without_gxx(tmp_path, monkeypatch)
    with pytest.raises(RuntimeError, match="no such header"):
        build.build()
    assert os.path.exists(build.LIB)


def test_the_command_line_builds_the_library(build, tmp_path, monkeypatch, capsys):
    without_gxx(tmp_path, monkeypatch)
    assert build.main([]) == 0
    out, err = capsys.readouterr()
    assert out.split() == [build.LIB] and os.path.exists(build.LIB)
    assert "no such header" in err


def test_the_library_does_not_need_torch(build, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)         # import torch raises ImportError
    with pytest.raises(RuntimeError, match="torch"):
        build.build()
    assert os.path.exists(build.LIB)


def test_a_missing_binding_does_not_rebuild_the_library(build, tmp_path, monkeypatch):
    without_gxx(tmp_path, monkeypatch)
    for _ in range(2):
        with pytest.raises(RuntimeError):
            build.build()
    assert sum("libra_gb300.so" in x for x in build.log.read_text().split()) == 1


def test_the_binding_belongs_to_one_torch(build, tmp_path, monkeypatch):
    """It holds the layout of torch's tensors: another torch gets its own, and does not load this one."""
    bin_dir = tmp_path / "bin"
    bin_dir.mkdir()
    log = tmp_path / "g++.log"
    script(bin_dir / "g++", """
echo run >> "%s"
while [ $# -gt 1 ]; do
  if [ "$1" = -o ]; then : > "$2"; fi
  shift
done
""" % log)
    monkeypatch.setenv("PATH", str(bin_dir) + os.pathsep + os.environ["PATH"])
    for _ in range(2):
        build.build()
    assert log.read_text().split() == ["run"]
    monkeypatch.setattr(torch, "__version__", "2.0.0+other")
    build.build()
    assert log.read_text().split() == ["run", "run"]


def test_the_package_does_not_load_another_torchs_binding(ralib, monkeypatch):
    ralib.native()
    monkeypatch.setattr(ralib, "_native", None)
    monkeypatch.setattr(torch, "__version__", "2.0.0+other")
    with pytest.raises(RuntimeError, match="not built"):
        ralib.native()
