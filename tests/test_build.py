"""What build.build() compiles and links, with the compilers replaced by a record
of their commands (nothing is compiled here)."""
import os
import subprocess
import sys

import pytest
import torch

import bit_expert_ffn_route_b200
from bit_expert_ffn_route_b200 import build, moe

TICK = 1_700_000_000


class Tree:
    """A source tree of one kernel file and the binding; compilers that write their output at the time `now`."""

    def __init__(self, root, monkeypatch):
        for name in ("csrc", "include", "_build"):
            (root / name).mkdir()
        self.now, self.ran, self.fails = TICK, [], ()
        self.files = {"cu": root / "csrc" / "a.cu", "h": root / "include" / "a.h", "cpp": root / "csrc" / "binding.cpp"}
        for f in self.files.values():
            self.touch(f)
        for name, at in dict(CSRC="csrc", INCLUDE="include", BUILD="_build", LIB="libmoe.so", OPS="_ops.so",
                             OPS_SRC="csrc/binding.cpp", OPS_FOR="_build/_ops.for").items():
            monkeypatch.setattr(build, name, str(root / at))
        monkeypatch.setattr(build.subprocess, "run", self.run)

    def touch(self, f):
        with open(f, "w") as out:
            out.write("x")
        os.utime(f, (self.now, self.now))

    def run(self, cmd, **_):
        out = os.path.basename(cmd[cmd.index("-o") + 1])
        self.ran.append(out)
        if out in self.fails:
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        self.touch(cmd[cmd.index("-o") + 1])
        return subprocess.CompletedProcess(cmd, 0, "", "")

    def build(self, **kw):
        self.ran = []
        build.build(**kw)
        return self.ran


@pytest.fixture
def tree(tmp_path, monkeypatch):
    return Tree(tmp_path, monkeypatch)


def test_what_is_newer_is_built_again(tree):
    assert tree.build() == ["a.o", "libmoe.so", "_ops.so"]
    assert tree.build() == []
    tree.now += 1
    tree.touch(tree.files["cpp"])
    assert tree.build() == ["_ops.so"]
    assert tree.build(force=True) == ["a.o", "libmoe.so", "_ops.so"]


def test_every_object_that_is_built_is_linked(tree):
    """Also where the file system's clock shows it no younger than the library: built in the library's own tick."""
    tree.now += 5
    tree.build()
    os.remove(os.path.join(build.BUILD, "a.o"))
    assert tree.build()[:2] == ["a.o", "libmoe.so"]


@pytest.mark.parametrize("how", ["compile error", "no compiler"])
def test_without_the_extension_module(tree, how, monkeypatch):
    """libmoe.so is built all the same, with a warning; the calls of moe_ops.h raise at their first use, and an
    extension module of older sources does not stay."""
    tree.build()
    tree.now += 1
    for f in tree.files.values():
        tree.touch(f)
    if how == "compile error":
        tree.fails = ("_ops.so",)
    else:
        monkeypatch.setattr(build, "_ops_command", lambda: (_ for _ in ()).throw(FileNotFoundError("g++")))
    with pytest.warns(RuntimeWarning, match="_ops.so was not built"):
        assert build.build() == build.LIB
    assert not os.path.exists(build.OPS) and os.path.getmtime(build.LIB) == tree.now
    with pytest.warns(RuntimeWarning):          # tried again by the next build
        build.build()


def test_a_call_without_the_extension_module(monkeypatch):
    """The import fails (None in sys.modules) as it does where the file is missing."""
    monkeypatch.setattr(moe, "lib", lambda: None)
    monkeypatch.setitem(sys.modules, "bit_expert_ffn_route_b200._ops", None)
    monkeypatch.delattr(bit_expert_ffn_route_b200, "_ops", raising=False)
    with pytest.raises(RuntimeError, match="_ops.so is missing"):
        moe.__getattr__("moe_permute")


def test_the_extension_module_is_built_for_one_torch(tree, monkeypatch):
    """Another torch: built again, although no source is newer."""
    assert "_ops.so" in tree.build()
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert tree.build() == ["_ops.so"]
    assert tree.build() == []


def test_the_extension_module_loads_with_its_torch_alone():
    """With another version in its place the import fails, and a call says what to do; with its own it works."""
    build.build()
    code = ("import torch\n{}\nfrom bit_expert_ffn_route_b200 import moe\ntry: moe.moe_permute\n"
            "except RuntimeError as e: print('refused', e, e.__cause__)\nelse: print('loaded')")
    for change, want in (("", "loaded"), ("torch.__version__ = '2.99.0'", "refused")):
        r = subprocess.run([sys.executable, "-c", code.format(change)], capture_output=True, text=True, cwd=build.ROOT)
        assert r.returncode == 0 and r.stdout.startswith(want), (r.stdout, r.stderr)
    assert "build --force" in r.stdout and "not 2.99.0" in r.stdout
