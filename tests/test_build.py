"""What build.py makes with and without torch, its compiles and links replaced by ones that
only write their outputs (CPU only)."""
import os
import subprocess
import sys

import pytest
import torch

from dense_gemm_16_amd import build


@pytest.fixture
def runs(monkeypatch, tmp_path):
    """The commands of a build into `tmp_path`."""
    commands = []

    def run(cmd, **kw):
        commands.append(cmd)
        if "-o" in cmd:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write("built")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build, "_compile", lambda unit, force: str(tmp_path / (unit[1] + ".o")))
    monkeypatch.setattr(build.subprocess, "run", run)
    for name, file in (("BUILD", "objects"), ("LIB", "libmigemm.so"), ("BINDING", "_binding.so"),
                       ("RESOURCES", "kernel_resources.json")):
        monkeypatch.setattr(build, name, str(tmp_path / file))
    return commands


def compiles(commands):
    return [c for c in commands if any(a.endswith("binding.cpp") for a in c)]


def test_without_torch(runs, monkeypatch, capsys):
    """The C library and its kernels' figures, and no binding, not an older one either."""
    monkeypatch.setitem(sys.modules, "torch", None)
    with open(build.BINDING, "w") as f:
        f.write("older")
    assert build.build(force=False) == build.LIB
    assert os.path.exists(build.LIB) and os.path.exists(build.RESOURCES)
    assert not os.path.exists(build.BINDING) and not compiles(runs)
    assert "torch is not installed" in capsys.readouterr().err


def test_the_binding_goes_by_the_installed_torch(runs, monkeypatch):
    build.build(force=False)
    assert os.path.exists(build.BINDING) and len(compiles(runs)) == 1
    flag = f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"
    assert flag in compiles(runs)[0]
    build.build(force=False)  # nothing has changed
    assert len(compiles(runs)) == 1
    monkeypatch.setattr(torch, "__version__", "another")
    build.build(force=False)
    assert len(compiles(runs)) == 2
    monkeypatch.setattr(torch, "compiled_with_cxx11_abi", lambda: flag.endswith("0"))
    build.build(force=False)
    assert len(compiles(runs)) == 3 and flag not in compiles(runs)[2]


def test_a_binding_that_does_not_compile(runs, monkeypatch):
    """Its error comes after the C library and the figures are whole."""
    fake = build.subprocess.run

    def run(cmd, **kw):
        if compiles([cmd]):
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        return fake(cmd, **kw)

    monkeypatch.setattr(build.subprocess, "run", run)
    with pytest.raises(RuntimeError, match="no such header"):
        build.build(force=False)
    assert os.path.exists(build.LIB) and os.path.exists(build.RESOURCES)
