"""The build's bookkeeping, with a stand-in for nvcc (no CUDA toolkit or GPU needed)."""
import os
import sys

import pytest

from gated_delta_rule_89_b200 import build as gbuild

# Compiles to its own flags, links to what its objects hold.
NVCC = """#!%s
import sys
a = sys.argv[1:]
out = a[a.index("-o") + 1]
if "-c" in a:
    text = a[-1].rsplit("/", 1)[1] + (" with -DLOUD" if "-DLOUD" in a else "") + "\\n"
else:
    text = "".join(open(p).read() for p in a[a.index("-o") + 2:])
open(out, "w").write(text)
""" % sys.executable


@pytest.fixture
def tree(tmp_path, monkeypatch):
    pkg = tmp_path / "pkg"
    (pkg / "csrc").mkdir(parents=True)
    (tmp_path / "include").mkdir()
    (tmp_path / "include" / "gdr.h").write_text("")
    for n in ("a.cu", "b.cu"):
        (pkg / "csrc" / n).write_text("")
    nvcc = tmp_path / "nvcc"
    nvcc.write_text(NVCC)
    nvcc.chmod(0o755)
    monkeypatch.setenv("NVCC", str(nvcc))
    monkeypatch.setattr(gbuild, "PKG", str(pkg))
    monkeypatch.setattr(gbuild, "ROOT", str(tmp_path))
    monkeypatch.setattr(gbuild, "LIB", str(pkg / "lib.so"))
    monkeypatch.setattr(gbuild, "OBJ", str(pkg / "_build"))
    return pkg


def touch(path, ahead):
    t = os.path.getmtime(gbuild.LIB) + ahead
    os.utime(path, (t, t))


def test_objects_of_other_flags_are_not_linked(tree):
    """A plain rebuild after one with extra flags holds none of its objects."""
    gbuild.build()
    gbuild.build(force=True, extra=["-DLOUD"])
    assert (tree / "lib.so").read_text() == "a.cu with -DLOUD\nb.cu with -DLOUD\n"
    touch(tree / "csrc" / "a.cu", 2)
    gbuild.build()
    assert (tree / "lib.so").read_text() == "a.cu\nb.cu\n"


def test_only_what_changed_is_compiled(tree):
    gbuild.build()
    before = {n: os.path.getmtime(tree / "_build" / n) for n in ("a.cu.o", "b.cu.o")}
    for n in before:
        os.utime(tree / "_build" / n, (before[n] + 5, before[n] + 5))
    touch(tree / "csrc" / "a.cu", 10)
    gbuild.build()
    assert os.path.getmtime(tree / "_build" / "b.cu.o") == before["b.cu.o"] + 5
    assert os.path.getmtime(tree / "_build" / "a.cu.o") != before["a.cu.o"] + 5
