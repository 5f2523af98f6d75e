"""The build: which steps depend on which.  The compilers are stand-ins that write what they are asked for, so
nothing is compiled here.  libcowa.so needs neither torch nor g++; _binding.so, which is built against the
installed torch, follows that torch and never stands half-written."""

import os
import stat
import sys

import pytest

from structured_sparse_attention_cowa_b200 import build as cbuild


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Outputs under tmp_path; nvcc and g++ write their command into the file after -o."""
    for name in ("nvcc", "g++"):
        exe = tmp_path / "bin" / name
        exe.parent.mkdir(exist_ok=True)
        exe.write_text("#!/bin/sh\nfor a in \"$@\"; do [ \"$p\" = -o ] && out=$a; p=$a; done\necho \"$0 $@\" > \"$out\"\n")
        exe.chmod(exe.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("PATH", f"{tmp_path / 'bin'}:{os.environ['PATH']}")
    monkeypatch.setenv("NVCC", str(tmp_path / "bin" / "nvcc"))
    monkeypatch.setattr(cbuild, "BUILD", str(tmp_path / "_build"))
    for name in ("LIB", "LIB_DEBUG", "BINDING"):
        monkeypatch.setattr(cbuild, name, str(tmp_path / os.path.basename(getattr(cbuild, name))))
    return tmp_path


def fail(exe):
    exe.write_text("#!/bin/sh\nfor a in \"$@\"; do [ \"$p\" = -o ] && out=$a; p=$a; done\necho half > \"$out\"\nexit 1\n")


@pytest.mark.parametrize("debug", [False, True])
def test_the_library_is_linked_where_the_binding_cannot_be_built(tree, debug):
    fail(tree / "bin" / "g++")
    with pytest.raises(RuntimeError, match="binding"):
        cbuild.build(debug=debug)
    assert os.path.exists(cbuild.LIB_DEBUG if debug else cbuild.LIB)


def test_a_machine_without_torch_gets_the_library(tree, monkeypatch, capfd):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert cbuild.build() == cbuild.LIB and os.path.exists(cbuild.LIB)
    assert not os.path.exists(cbuild.BINDING)
    assert "torch" in capfd.readouterr().err  # what was left out, and why
