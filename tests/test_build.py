"""What build() compiles and when, with the compilers replaced by a recorder."""
import os
import subprocess

import pytest
import torch

from verify_gated_gqa_gb300 import build as build_mod


class Commands:
    """Stands in for subprocess.run: notes each command's program and writes its output file."""

    def __init__(self):
        self.ran, self.failing = [], None

    def __call__(self, cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        self.ran.append((os.path.basename(cmd[0]), os.path.basename(out)))
        ok = self.failing is None or self.failing not in os.path.basename(out)
        if ok:
            with open(out, "w"):
                pass
        return subprocess.CompletedProcess(cmd, 0 if ok else 1, "", "")

    def take(self):
        ran, self.ran = self.ran, []
        return sorted(ran)


@pytest.fixture
def commands(monkeypatch, tmp_path):
    c = Commands()
    monkeypatch.setattr(build_mod.subprocess, "run", c)
    monkeypatch.setattr(build_mod, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build_mod, "LIB", str(tmp_path / "libga_attn.so"))
    monkeypatch.setattr(build_mod, "NATIVE", str(tmp_path / "_native.so"))
    return c


NATIVE_STEPS = [("g++", "_native.so"), ("g++", "ga_native.o")]


def test_native_module_follows_torch_and_python(commands, monkeypatch):
    """Built once, and again when the torch or the Python that it was compiled against changes."""
    build_mod.build()
    first = commands.take()
    assert set(NATIVE_STEPS) <= set(first) and ("nvcc", "libga_attn.so") in first
    build_mod.build()
    assert commands.take() == []
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    build_mod.build()
    assert commands.take() == NATIVE_STEPS
    build_mod.build()
    assert commands.take() == []
    real = build_mod.sysconfig.get_config_var
    monkeypatch.setattr(build_mod.sysconfig, "get_config_var",
                        lambda name: "other" if name == "SOABI" else real(name))
    build_mod.build()
    assert commands.take() == NATIVE_STEPS


def test_library_is_built_without_torch(commands, monkeypatch, capsys):
    """The C-ABI library needs nvcc alone; the native module is left out, and said to be."""
    monkeypatch.setitem(build_mod.sys.modules, "torch", None)   # import torch raises ImportError
    assert build_mod.build() == build_mod.LIB
    ran = commands.take()
    assert ("nvcc", "libga_attn.so") in ran and not any(p == "g++" for p, _ in ran)
    assert "_native.so" in capsys.readouterr().err


def test_library_is_linked_before_the_native_module_fails(commands):
    commands.failing = "ga_native"
    with pytest.raises(RuntimeError):
        build_mod.build()
    assert ("nvcc", "libga_attn.so") in commands.take()
    commands.failing = None
    build_mod.build()
    assert commands.take() == NATIVE_STEPS
