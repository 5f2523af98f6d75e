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


def test_the_binding_follows_the_installed_torch(tree, monkeypatch):
    import torch

    cbuild.build()
    first = os.stat(cbuild.BINDING).st_mtime_ns
    os.utime(cbuild.BINDING, ns=(first, first + 10**12))  # newer than any source
    (tree / "bin" / "g++").write_text((tree / "bin" / "g++").read_text().replace("echo \"", "echo \"again "))
    cbuild.build()
    assert "again" not in open(cbuild.BINDING).read()  # nothing has changed
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    cbuild.build()
    assert "again" in open(cbuild.BINDING).read()


def test_a_binding_of_unknown_origin_is_built_again(tree):
    """A file that this build did not write, newer than its source: there at the start, or put in place later."""
    for _ in range(2):
        with open(cbuild.BINDING, "w") as f:
            f.write("something")
        later = os.stat(cbuild.BINDING).st_mtime_ns + 10**12
        os.utime(cbuild.BINDING, ns=(later, later))
        cbuild.build()
        assert "g++" in open(cbuild.BINDING).read()


def test_a_binding_that_fails_to_build_leaves_no_half_of_itself(tree):
    """What g++ leaves of a build that fails is not imported, and the old file stays whole until the new one is
    there."""
    good = (tree / "bin" / "g++").read_text()
    fail(tree / "bin" / "g++")
    with pytest.raises(RuntimeError, match="binding"):
        cbuild.build()
    assert not os.path.exists(cbuild.BINDING)
    (tree / "bin" / "g++").write_text(good)
    cbuild.build()
    old = open(cbuild.BINDING).read()
    fail(tree / "bin" / "g++")
    src_newer = os.stat(os.path.join(cbuild.CSRC, "binding.cpp")).st_mtime_ns - 10**12
    os.utime(cbuild.BINDING, ns=(src_newer, src_newer))
    with pytest.raises(RuntimeError, match="binding"):
        cbuild.build()
    assert open(cbuild.BINDING).read() == old
