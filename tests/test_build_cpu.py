"""What build.py compiles and when (no compiler runs here)."""
import os
import sys

import pytest

from diffusion_decoding_step_b200 import build


@pytest.fixture
def calls(tmp_path, monkeypatch):
    """The commands build.py runs; each leaves its output file behind.  Nothing in the tree is
    written."""
    made = []

    def run(cmd, check):
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        made.append(os.path.basename(out).removesuffix(".tmp"))

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libdllm.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_paged_torch.so"))
    return made


def test_library_comes_first_and_both_are_built_once(calls):
    assert build.build() == build.LIB
    assert calls == ["libdllm.so", "_paged_torch.so"]
    assert build.build() == build.LIB
    assert len(calls) == 2
    build.build(force=True)
    assert len(calls) == 4


def test_library_needs_no_torch(calls, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)     # import torch: ImportError
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert calls == ["libdllm.so"]
    assert "_paged_torch.so is left out" in capsys.readouterr().err


def test_library_needs_no_python_headers(calls, tmp_path, monkeypatch, capsys):
    import sysconfig
    monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert build.build() == build.LIB
    assert calls == ["libdllm.so"]
    assert "Python.h" in capsys.readouterr().err


def test_a_failing_binding_is_an_error_but_leaves_the_library(calls, monkeypatch):
    run = build.subprocess.run

    def fails(cmd, check):
        if build.BINDING + ".tmp" in cmd:
            raise build.subprocess.CalledProcessError(1, cmd)
        run(cmd, check)

    monkeypatch.setattr(build.subprocess, "run", fails)
    with pytest.raises(build.subprocess.CalledProcessError):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)


def test_another_torch_means_another_binding(calls, monkeypatch):
    import torch
    build.build()
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    build.build()
    assert calls == ["libdllm.so", "_paged_torch.so", "_paged_torch.so"]
    build.build()
    assert len(calls) == 3
    os.remove(build.BINDING + ".made_for")      # built by something that left no note
    build.build()
    assert len(calls) == 4
