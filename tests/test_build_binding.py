"""The build of the native binding: it is linked again whenever it is older than what it is made of."""
import os
import subprocess

import pytest

from exact_tiled_attention_21_gb300 import _build


class Tools:
    """Stands in for nvcc and g++: an output file per command, which holds the time step at which it was made."""

    def __init__(self, monkeypatch):
        self.step, self.fail, self.ran = 1000, (), []
        monkeypatch.setattr(_build.subprocess, "run", self.run)

    def run(self, cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        self.ran.append(os.path.basename(out).split(".tmp")[0])
        if any(os.path.basename(out).startswith(f) for f in self.fail):
            return subprocess.CompletedProcess(cmd, 1, "", "planted")
        with open(out, "w") as f:
            f.write(str(self.step))
        os.utime(out, (self.step, self.step))
        return subprocess.CompletedProcess(cmd, 0, "", "")

    def build(self, step, fail=()):
        self.step, self.fail, self.ran = step, fail, []
        _build.build()
        return self.ran


@pytest.fixture
def tree(tmp_path, monkeypatch):
    csrc, inc = tmp_path / "pkg" / "csrc", tmp_path / "include"
    csrc.mkdir(parents=True)
    inc.mkdir()
    for f in ("a.cu", "fa_torch.cpp", "x.cuh"):
        (csrc / f).write_text("")
    (inc / "fa.h").write_text("")
    at = {"HERE": tmp_path / "pkg", "CSRC": csrc, "ROOT": tmp_path, "LIB": tmp_path / "pkg" / "lib.so",
          "TORCH_LIB": tmp_path / "pkg" / "binding.so", "BUILD": tmp_path / "_build",
          "TORCH_OBJ": tmp_path / "_build" / "fa_torch.o"}
    for name, path in at.items():
        monkeypatch.setattr(_build, name, str(path))
    monkeypatch.setattr(_build, "SOURCES", ["a.cu"])

    def touch(name, step):
        os.utime(csrc / name if (csrc / name).exists() else inc / name, (step, step))
    for f in ("a.cu", "fa_torch.cpp", "x.cuh", "fa.h"):
        touch(f, 500)
    return Tools(monkeypatch), touch, at


def test_binding_links_after_a_build_that_failed_elsewhere(tree):
    tools, touch, at = tree
    assert set(tools.build(1000)) == {"a.o", "fa_torch.o", "lib.so", "binding.so"}
    assert tools.build(1001) == []
    for part in ("a.o", "lib.so", "binding.so"):            # where the build stops after the binding was compiled
        touch("fa.h", tools.step + 10)
        with pytest.raises(RuntimeError):
            tools.build(tools.step + 20, fail=(part,))
        stale = at["TORCH_LIB"].read_text()
        again = tools.build(tools.step + 30)
        assert "binding.so" in again and at["TORCH_LIB"].read_text() != stale, part
        assert tools.build(tools.step + 1) == []


def test_binding_is_compiled_again_for_another_torch(tree, monkeypatch):
    import torch
    tools, touch, at = tree
    tools.build(1000)
    monkeypatch.setattr(torch, "__version__", "0.0.other")
    with pytest.raises(RuntimeError):
        tools.build(1010, fail=("binding.so",))
    assert "binding.so" in tools.build(1020)
    assert tools.build(1030) == []
