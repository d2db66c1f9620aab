"""What the build makes, and what it needs for it (CPU only, no compiler is run)."""
import os
import subprocess
import sys

import pytest

from speculative_decoding_verification_51_gb300 import build as B


@pytest.fixture
def commands(tmp_path, monkeypatch):
    """The build in an empty folder with compilers that only write their output."""
    done = []

    def run(cmd, **kw):
        done.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(B, "BUILD", str(tmp_path))
    monkeypatch.setattr(B.subprocess, "run", run)
    return done


def outputs(done):
    return sorted(os.path.basename(c[c.index("-o") + 1]).split(".")[0].split("_" + B.platform.machine())[0] for c in done if "-shared" in c)


def test_without_torch_there_is_the_library(commands, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)        # import torch: ImportError
    assert B.build() == B.lib_path() and os.path.exists(B.lib_path())
    assert outputs(commands) == ["libspecverify"]
    assert not any("torch_ops" in a or a.startswith("-ltorch") for c in commands for a in c)
    del commands[:]
    B.build()
    assert B.up_to_date() and commands == []
    B.build(force=True)
    assert outputs(commands) == ["libspecverify"]


def test_each_is_made_when_its_own_inputs_change(commands):
    B.build()
    assert outputs(commands) == ["libspecverify", "specverify_torch"]
    del commands[:]
    B.build()
    assert commands == []
    os.utime(B.ops_path(), (1, 1))                          # older than its source
    B.build()
    assert outputs(commands) == ["specverify_torch"]
    del commands[:]
    os.utime(B.lib_path(), (1, 1))
    B.build()
    assert outputs(commands) == ["libspecverify"]
    del commands[:]
    os.remove(B.ops_path())
    assert not B.up_to_date()


def test_the_library_does_not_wait_for_the_module(commands, monkeypatch):
    run = B.subprocess.run

    def fails(cmd, **kw):
        if any("torch_ops.cpp" in str(a) for a in cmd):
            return subprocess.CompletedProcess(cmd, 1, "", "no headers")
        return run(cmd, **kw)

    monkeypatch.setattr(B.subprocess, "run", fails)
    with pytest.raises(RuntimeError, match="torch_ops.cpp"):
        B.build()
    assert os.path.exists(B.lib_path()) and not os.path.exists(B.ops_path())
