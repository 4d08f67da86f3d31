"""The build script on a host without PyTorch, or without a C++ compiler: the library is built, the native
argument checks are left out with a word on why, and an old file of theirs goes."""
import os
import sys

import pytest

import prefill_only_cascade_gb300.build as build


@pytest.fixture
def calls(tmp_path, monkeypatch):
    """Another place for the file, with one from before in it."""
    path = tmp_path / "_paged_calls.so"
    path.write_bytes(b"old")
    monkeypatch.setattr(build, "CALLS", str(path))
    return path


@pytest.mark.parametrize("how", ["hidden", "missing", "no compiler"])
def test_left_out_with_a_reason(how, calls, monkeypatch, capsys):
    if how == "hidden":
        monkeypatch.setitem(sys.modules, "torch", None)
    elif how == "missing":
        monkeypatch.delitem(sys.modules, "torch", raising=False)
        monkeypatch.setattr(sys, "path", [])
        monkeypatch.setattr(sys, "path_importer_cache", {})
    else:
        monkeypatch.setenv("PATH", os.devnull)
    assert build.build_calls("/usr/local/cuda/bin/nvcc") is None
    assert "not built" in capsys.readouterr().err
    assert not calls.exists()


def test_library_is_linked_without_pytorch(calls, tmp_path, monkeypatch):
    """The whole of build(), the compiler's runs replaced by files of the names that they make."""
    monkeypatch.setitem(sys.modules, "torch", None)
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libquail.so"))
    monkeypatch.setattr(build, "nvcc_path", lambda: "nvcc")

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def run(cmd, **_):
        with open(cmd[cmd.index("-o") + 1], "wb") as f:
            f.write(b"made")
        return Done()

    monkeypatch.setattr(build.subprocess, "run", run)
    assert build.build() == str(tmp_path / "libquail.so")
    assert (tmp_path / "libquail.so").read_bytes() == b"made" and not calls.exists()
