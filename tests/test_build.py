"""build.py with the compilers stood in for (no GPU, nothing compiled): what is
built when, and in which order."""
import os
import subprocess
import sys

import pytest

from orthogonal_equivalence_b200 import build as pbuild


@pytest.fixture
def compilers(monkeypatch, tmp_path):
    """Paths in tmp_path and a subprocess.run that writes each command's -o file; returns the outputs' names."""
    made = []

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        made.append(os.path.basename(out).split(".so")[0])
        with open(out, "wb") as f:
            f.write(" ".join(cmd).encode())
        return subprocess.CompletedProcess(cmd, 0, "", "")

    for name in ("LIB", "LIB_DEBUG", "TENSORS"):
        monkeypatch.setattr(pbuild, name, str(tmp_path / os.path.basename(getattr(pbuild, name))))
    monkeypatch.setattr(pbuild.subprocess, "run", run)
    return made


def test_the_library_is_built_before_the_extension(compilers):
    assert pbuild.build() == pbuild.LIB
    assert compilers == ["libpoetx", "_tensors"]
    pbuild.build(debug=True)
    assert compilers == ["libpoetx", "_tensors", "libpoetx_debug"]
    pbuild.build()
    assert len(compilers) == 3


def test_the_library_is_built_where_torch_is_missing(compilers, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)      # import torch raises ImportError
    assert pbuild.build() == pbuild.LIB and os.path.exists(pbuild.LIB)
    assert compilers == ["libpoetx"]
    assert "_tensors.so" in capsys.readouterr().err


def test_an_extension_that_does_not_compile_leaves_the_library(compilers, monkeypatch):
    run = pbuild.subprocess.run

    def fails(cmd, **kw):
        return run(cmd, **kw) if "_tensors" not in cmd[cmd.index("-o") + 1] else subprocess.CompletedProcess(cmd, 1, "", "no")

    monkeypatch.setattr(pbuild.subprocess, "run", fails)
    with pytest.raises(RuntimeError, match="_tensors.so"):
        pbuild.build()
    assert os.path.exists(pbuild.LIB)


def test_the_extension_follows_torch_and_python(compilers, monkeypatch):
    import torch
    pbuild.build_tensors()
    pbuild.build_tensors()
    assert compilers == ["_tensors"]
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    pbuild.build_tensors()
    pbuild.build_tensors()
    assert compilers == ["_tensors"] * 2
    monkeypatch.setattr(sys.implementation, "cache_tag", "cpython-399")
    pbuild.build_tensors()
    assert compilers == ["_tensors"] * 3
