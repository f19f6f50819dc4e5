"""The build's rules for what it may reuse."""
import os
import subprocess
import time

import pytest


@pytest.fixture
def compiles(tmp_path, monkeypatch):
    """The front end's compile step with a recorded, empty compiler."""
    from block_sparse_attention_proxy_gb300 import build

    runs = []

    def run(cmd, **kw):
        runs.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build.subprocess, "run", run)

    def step(newest=0.0):
        before = len(runs)
        assert os.path.exists(build._compile_torch(newest))
        return len(runs) - before

    return step


def test_the_front_end_is_reused(compiles):
    assert [compiles(), compiles(), compiles()] == [1, 0, 0]
    assert compiles(newest=time.time() + 10) == 1  # a newer source


def test_the_front_end_is_rebuilt_for_another_torch(compiles, monkeypatch):
    import torch

    assert compiles() == 1
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert [compiles(), compiles()] == [1, 0]


def test_the_front_end_is_rebuilt_for_another_python(compiles, monkeypatch):
    import sysconfig

    assert compiles() == 1
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-299")
    assert [compiles(), compiles()] == [1, 0]


def test_a_failed_compile_leaves_nothing_to_reuse(compiles, monkeypatch):
    import torch
    from block_sparse_attention_proxy_gb300 import build

    assert compiles() == 1
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    good = build.subprocess.run
    monkeypatch.setattr(build.subprocess, "run",
                        lambda cmd, **kw: subprocess.CompletedProcess(cmd, 1, "", "no"))
    with pytest.raises(RuntimeError):
        compiles()
    monkeypatch.setattr(build.subprocess, "run", good)
    assert compiles() == 1


def test_a_front_end_that_does_not_load_says_why(monkeypatch, tmp_path):
    import sys

    from block_sparse_attention_proxy_gb300 import dense

    there, absent = tmp_path / "there.so", tmp_path / "absent.so"
    there.touch()
    monkeypatch.setattr(dense, "load", lambda: None)
    monkeypatch.setattr(dense, "_call", None)
    monkeypatch.setitem(sys.modules, "block_sparse_attention_proxy_gb300._dense_torch", None)
    monkeypatch.setattr(dense, "TORCH_LIB", str(there))
    with pytest.raises(RuntimeError, match="does not load: .*_dense_torch") as error:
        dense._load()
    assert "missing" not in str(error.value)
    monkeypatch.setattr(dense, "TORCH_LIB", str(absent))
    with pytest.raises(RuntimeError, match="is missing: build the library"):
        dense._load()
