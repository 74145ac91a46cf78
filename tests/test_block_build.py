"""What a build leaves behind (no compiler is run: the commands are answered
by a stand-in that writes their outputs)."""
import os
import subprocess

import pytest

from sparse_moe_routed_amd import build as B


class Compilers:
    """subprocess.run of the build: fails as told, else writes what -o names."""

    def __init__(self):
        self.failing = lambda cmd: False
        self.missing = ()

    def run(self, cmd, **kw):
        if os.path.basename(cmd[0]) in self.missing:
            raise FileNotFoundError(cmd[0])
        if self.failing(cmd):
            return subprocess.CompletedProcess(cmd, 1, "", "no")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("new")
        return subprocess.CompletedProcess(cmd, 0, "", "")


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """(stand-in, libmoe.so, _block.so) with an older build in place."""
    c = Compilers()
    monkeypatch.setattr(B.subprocess, "run", c.run)
    monkeypatch.setattr(B, "BUILD", str(tmp_path / "_build"))
    lib, binding = tmp_path / "libmoe.so", tmp_path / "_block.so"
    monkeypatch.setattr(B, "LIB", str(lib))
    monkeypatch.setattr(B, "BINDING", str(binding))
    which = B.shutil.which
    monkeypatch.setattr(B.shutil, "which", lambda n, *a, **k: None if n in c.missing else which(n, *a, **k))
    lib.write_text("old")
    binding.write_text("old")
    return c, lib, binding


def test_both_are_new(tree):
    c, lib, binding = tree
    assert B.build(verbose=False) == str(lib)
    assert lib.read_text() == binding.read_text() == "new"
    assert sorted(p.name for p in lib.parent.iterdir()) == ["_block.so", "_build", "libmoe.so"]


@pytest.mark.parametrize("what", ["hip source", "library link", "binding compile", "binding link"])
def test_a_failed_build_leaves_the_older_pair(tree, what):
    """Not a new library beside an old binding, nor the other way round."""
    c, lib, binding = tree
    out = lambda cmd: os.path.basename(cmd[cmd.index("-o") + 1])
    c.failing = {"hip source": lambda cmd: out(cmd) == "k_norm.hip.o",
                 "library link": lambda cmd: out(cmd).startswith("libmoe.so"),
                 "binding compile": lambda cmd: out(cmd) == "block_binding.o",
                 "binding link": lambda cmd: out(cmd).startswith("_block.so")}[what]
    with pytest.raises(RuntimeError):
        B.build(verbose=False)
    assert lib.read_text() == binding.read_text() == "old"


@pytest.mark.parametrize("gone", ["g++", "Python.h", "torch"])
def test_the_library_needs_only_hipcc(tree, gone, monkeypatch, capsys):
    """Where the binding cannot be built the C library still is, and no older
    binding stays beside it: the calls that need it then say so."""
    c, lib, binding = tree
    if gone == "g++":
        c.missing = ("g++",)
    elif gone == "Python.h":
        monkeypatch.setattr(B.sysconfig, "get_paths", lambda: {"include": str(lib.parent / "nowhere")})
        c.failing = lambda cmd: os.path.basename(cmd[0]) == "g++"
    else:
        monkeypatch.setitem(__import__("sys").modules, "torch", None)
    B.build(verbose=False)
    assert lib.read_text() == "new" and not binding.exists()
    assert gone in capsys.readouterr().err
