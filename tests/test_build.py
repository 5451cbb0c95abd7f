"""The C library builds where the operators' Python module cannot be compiled (no g++, no headers of
torch or Python), and only that module's calls fail then."""
import os
import subprocess
import warnings

import pytest
import torch

from gated_delta_rule_48_gb300 import binding as kb


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """A build of one small source, in a folder of its own, with nothing loaded."""
    src = tmp_path / "one.cu"
    src.write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(kb, "_sources", lambda: [str(src)])
    monkeypatch.setattr(kb, "_BUILD", str(tmp_path / "b"))
    monkeypatch.setattr(kb, "_LIB", str(tmp_path / "b" / "libkda.so"))
    monkeypatch.setattr(kb, "_EXT", str(tmp_path / "b" / "ext" / "kda_torch.so"))
    monkeypatch.setattr(kb, "load", lambda: None)
    monkeypatch.setattr(kb, "_extension", None)
    monkeypatch.setattr(kb, "_selected", None)
    return tmp_path


def no_compiler(monkeypatch):
    popen = subprocess.Popen

    def start(cmd, *args, **kwargs):
        if cmd[0] == "g++":
            raise FileNotFoundError(2, "No such file or directory", "g++")
        return popen(cmd, *args, **kwargs)
    monkeypatch.setattr(kb.subprocess, "Popen", start)


def no_headers(monkeypatch):
    monkeypatch.setattr(kb.sysconfig, "get_paths", lambda: {"include": "/nonexistent"})


@pytest.mark.parametrize("lacking", [no_compiler, no_headers])
def test_the_library_builds_without_the_module(elsewhere, monkeypatch, lacking):
    lacking(monkeypatch)
    os.makedirs(os.path.dirname(kb._EXT))
    with open(kb._EXT, "w") as f:  # of an older source: not to be loaded
        f.write("old")
    os.utime(kb._EXT, (1, 1))
    for _ in range(2):  # built, and up to date
        with pytest.warns(RuntimeWarning, match="operators' Python calls are not available"):
            path = kb.build()
        assert path == kb._LIB and os.path.exists(path)
    with pytest.raises(RuntimeError, match="kda_torch: compilation failed"):
        kb.kda_add_rms_norm(torch.zeros(2, 8), torch.zeros(8))


def test_a_library_that_does_not_compile_is_an_error(elsewhere, monkeypatch):
    no_compiler(monkeypatch)
    (elsewhere / "one.cu").write_text("this is no source\n")
    with pytest.raises(RuntimeError, match="nvcc failed"):
        kb.build()
    assert not os.path.exists(kb._LIB)


def test_the_library_is_there_where_warnings_are_errors(elsewhere, monkeypatch):
    no_compiler(monkeypatch)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(RuntimeWarning, match="operators' Python calls are not available"):
            kb.build()
    assert os.path.exists(kb._LIB)
