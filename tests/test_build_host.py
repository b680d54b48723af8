"""The build without its compilers: what is built when, and what a missing or
changed torch means for it."""
import os
import sys
import types

import pytest

from quantised_linear_layers_gb300 import build


@pytest.fixture
def fake(monkeypatch, tmp_path):
    """build in an empty folder with compilers that write empty files; returns the commands that were run."""
    run = []

    def subprocess_run(cmd, **kw):
        run.append(cmd)
        fail = fake_fail and cmd[0] == fake_fail[0]
        if not fail:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=1 if fail else 0, stdout="", stderr="no such header" if fail else "")

    fake_fail = []
    monkeypatch.setattr(build.subprocess, "run", subprocess_run)
    monkeypatch.setattr(build, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libqlinear.so"))
    monkeypatch.setattr(build, "TORCH_LIB", str(tmp_path / "_fp4.so"))
    return types.SimpleNamespace(run=run, fail=fake_fail, gxx=lambda: [c for c in run if c[0] == "g++"])


def test_both_are_built_once(fake):
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and os.path.exists(build.TORCH_LIB) and len(fake.gxx()) == 1
    n = len(fake.run)
    build.build()
    assert len(fake.run) == n


def test_the_library_needs_no_torch(fake, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.TORCH_LIB) and not fake.gxx()


def test_a_module_that_does_not_compile_is_reported_after_the_library(fake):
    fake.fail.append("g++")
    with pytest.raises(RuntimeError, match="no such header"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.TORCH_LIB)
    fake.fail.clear()
    build.build()
    assert os.path.exists(build.TORCH_LIB)


def test_another_torch_or_python_means_another_module(fake, monkeypatch):
    import torch
    build.build()
    assert len(fake.gxx()) == 1
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    build.build()
    assert len(fake.gxx()) == 2
    build.build()
    assert len(fake.gxx()) == 2
    monkeypatch.setattr(sys, "version", "4.0.0 (another build)")
    build.build()
    assert len(fake.gxx()) == 3
