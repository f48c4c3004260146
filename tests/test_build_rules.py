"""What a build compiles and links, on a tree of empty sources with a compiler
that only makes files."""
import os
import subprocess
import types

import pytest

from normalization_token_split_gb300 import _abi, _lib
from normalization_token_split_gb300 import build as nts_build


class Tree:
    def __init__(self, root, monkeypatch):
        self.root, self.now, self.broken, self.ran = root, 1000, set(), []
        for d in ("csrc", "include", "binding", "_build"):
            (root / d).mkdir()
        for name, path in (("CSRC", "csrc"), ("INCLUDE", "include"), ("BUILD", "_build"),
                           ("LIB", "_build/libnts.so"), ("BINDING", "binding/marshal.cpp"),
                           ("MARSHAL", "_build/marshal_nts.so")):
            monkeypatch.setattr(nts_build, name, str(root / path))
        monkeypatch.setattr(nts_build.subprocess, "run", self.run)
        self.touch("csrc/a.cu", "csrc/b.cu", "csrc/c.cpp", "csrc/x.cuh", "include/nts.h",
                   "binding/marshal.cpp")

    def touch(self, *names):
        for n in names:
            self.now += 10
            (self.root / n).touch()
            os.utime(self.root / n, (self.now, self.now))

    def run(self, cmd, **_):
        """A compiler: fails for sources in `broken`, else makes what -o names."""
        what = os.path.basename(cmd[cmd.index("-c") + 1]) if "-c" in cmd else "link " + (
            "marshal" if any("marshal" in c for c in cmd) else "lib")
        self.ran.append(what)
        if what in self.broken:
            return subprocess.CompletedProcess(cmd, 1, "", "broken")
        out = cmd[cmd.index("-o") + 1]
        self.now += 10
        open(out, "w").close()
        os.utime(out, (self.now, self.now))
        return subprocess.CompletedProcess(cmd, 0, "", "")

    def build(self, fails=False, **kw):
        self.ran = []
        if fails:
            with pytest.raises(RuntimeError):
                nts_build.build(**kw)
        else:
            nts_build.build(**kw)
        return sorted(self.ran)


@pytest.fixture
def tree(tmp_path, monkeypatch):
    # one job at a time: the times of what it makes stay in order
    one = types.SimpleNamespace(cpu_count=lambda: 1)
    monkeypatch.setattr(nts_build.os, "cpu_count", one.cpu_count)
    return Tree(tmp_path, monkeypatch)


ALL = ["a.cu", "b.cu", "c.cpp", "link lib", "link marshal", "marshal.cpp"]


def test_only_what_changed(tree):
    assert tree.build() == ALL
    assert tree.build() == []
    assert tree.build(force=True) == ALL
    tree.touch("csrc/b.cu")
    assert tree.build() == ["b.cu", "link lib"]
    tree.touch("binding/marshal.cpp")
    assert tree.build() == ["link marshal", "marshal.cpp"]
    tree.touch("include/nts.h")
    assert tree.build() == ALL


def test_a_failed_unit_leaves_nothing_unlinked(tree):
    """The declarations change and one unit does not compile: the others' objects
    are new, and the run that mends it links them all."""
    tree.build()
    tree.touch("include/nts.h")
    tree.broken = {"b.cu"}
    tree.build(fails=True)
    tree.broken = set()
    assert tree.build() == ["b.cu", "link lib", "link marshal"]
    assert tree.build() == []


def test_a_failed_binding_leaves_the_library_current(tree):
    tree.build()
    tree.touch("csrc/a.cu", "binding/marshal.cpp")
    tree.broken = {"marshal.cpp"}
    tree.build(fails=True)
    lib, obj = (os.path.getmtime(tree.root / "_build" / n) for n in ("libnts.so", "a.cu.o"))
    tree.broken = set()
    ran = tree.build()
    assert {"link marshal", "marshal.cpp"} <= set(ran) and "a.cu" not in ran
    assert "link lib" in ran or lib > obj


def test_a_failed_link_is_tried_again(tree):
    tree.build()
    for broken, source in (("link lib", "csrc/a.cu"), ("link marshal", "binding/marshal.cpp")):
        tree.touch(source)
        tree.broken = {broken}
        tree.build(fails=True)
        tree.broken = set()
        assert broken in tree.build()
        assert tree.build() == []


def test_the_extension_is_of_one_python_and_one_torch(monkeypatch):
    import torch

    name = os.path.basename(_lib.MARSHAL_PATH)
    assert _lib.MARSHAL_PATH == nts_build.MARSHAL and name == _abi.marshal_name()
    assert _abi.torch_version() == torch.__version__ and torch.__version__ in name
    monkeypatch.setattr(_abi, "torch_version", lambda: "0.0")
    assert _abi.marshal_name() != name
    monkeypatch.undo()
    monkeypatch.setattr(_abi.sysconfig, "get_config_var", lambda _: "cpython-399")
    assert _abi.marshal_name() != name


def test_another_abi_s_extension_is_neither_kept_nor_loaded(tree, monkeypatch):
    tree.build()
    other = str(tree.root / "_build" / "marshal_nts.another.so")
    monkeypatch.setattr(nts_build, "MARSHAL", other)
    assert tree.build() == ["link marshal", "marshal.cpp"]
    assert os.path.exists(other)
    monkeypatch.setattr(_lib, "_marshal", None)
    monkeypatch.setattr(_lib, "MARSHAL_PATH", str(tree.root / "_build" / "marshal_nts.third.so"))
    with pytest.raises(RuntimeError, match="this torch is not built"):
        _lib.marshal()


@pytest.mark.parametrize("lacks", ["torch", "torch's headers", "Python's headers"])
def test_the_library_is_built_without_what_the_extension_needs(tree, monkeypatch, capsys, lacks):
    if lacks == "torch":
        monkeypatch.setattr(nts_build, "torch_dir", lambda: None)
    elif lacks == "torch's headers":
        monkeypatch.setattr(nts_build, "torch_dir", lambda: str(tree.root))
    else:
        monkeypatch.setattr(nts_build.sysconfig, "get_paths",
                            lambda: {"include": str(tree.root / "none")})
    assert tree.build() == ["a.cu", "b.cu", "c.cpp", "link lib"]
    assert "is missing" in capsys.readouterr().err
    monkeypatch.undo()
    assert not (tree.root / "_build" / "marshal_nts.so").exists()
