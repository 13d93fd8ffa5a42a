"""The build's idea of what is up to date, on a small tree of its own (build.py with two tiny units): a tree that was
copied or moved with its objects, edited headers, and compilations that fail."""
import importlib.util
import os
import shutil
import subprocess
import time

import pytest

from precision_flashattention_numerics_gb300 import build as real


def load(root):
    spec = importlib.util.spec_from_file_location("build_of_" + os.path.basename(root), os.path.join(root, "pkg", "build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def write(path, text, age=0):
    os.makedirs(os.path.dirname(path), exist_ok=True)
    with open(path, "w") as f:
        f.write(text)
    t = time.time() - age
    os.utime(path, (t, t))


@pytest.fixture(scope="module")
def built(tmp_path_factory):
    root = str(tmp_path_factory.mktemp("tree") / "a")
    write(f"{root}/include/api.h", "#define API 1\n", 100)
    write(f"{root}/pkg/csrc/one.cuh", "#include \"two.cuh\"\n", 100)
    write(f"{root}/pkg/csrc/two.cuh", "#define TWO 2\n", 100)
    write(f"{root}/pkg/csrc/a.cu", "#include \"../../include/api.h\"\n#include \"one.cuh\"\nextern \"C\" int a() { return API + TWO; }\n", 100)
    write(f"{root}/pkg/csrc/b.cu", "#include \"two.cuh\"\nextern \"C\" int b() { return TWO; }\n", 100)
    shutil.copy(real.__file__, f"{root}/pkg/build.py")
    os.utime(f"{root}/pkg/build.py", (time.time() - 100,) * 2)
    m = load(root)
    m.LIB = m.LIB.replace("libpasa.so", "lib.so")
    m.build()
    return root


def tree(built, to, copy=shutil.copytree):
    copy(built, to)
    m = load(to)
    m.LIB = m.LIB.replace("libpasa.so", "lib.so")
    return m


def touch(path):
    t = time.time() + 5
    os.utime(path, (t, t))


SOURCES = {"include/api.h": ["a"], "pkg/csrc/one.cuh": ["a"], "pkg/csrc/two.cuh": ["a", "b"], "pkg/csrc/a.cu": ["a"], "pkg/csrc/b.cu": ["b"],
           "pkg/build.py": ["a", "b"]}


@pytest.mark.parametrize("source", SOURCES)
def test_edits_in_a_copied_tree_are_seen(built, tmp_path, source):
    m = tree(built, str(tmp_path / "copy"))
    assert not m.needs_build()
    touch(str(tmp_path / "copy" / source))
    assert m.needs_build() and [u for u in ("a", "b") if m._stale(u)] == SOURCES[source]


def test_what_lies_in_the_first_tree_plays_no_part(built, tmp_path):
    m = tree(built, str(tmp_path / "copy"))
    first = os.path.join(built, "pkg", "csrc", "two.cuh")
    before = os.stat(first)
    touch(first)
    try:
        assert not m.needs_build()
    finally:
        os.utime(first, (before.st_atime, before.st_mtime))
    assert str(tmp_path) not in open(os.path.join(built, "pkg", "_build", "a.d")).read()


def test_dependency_files_of_another_tree_do_not_count(built, tmp_path):
    """With absolute paths of another tree, as they were written once, or with none, an object is made again."""
    m = tree(built, str(tmp_path / "copy"))
    d = os.path.join(m.OBJ, "a.d")
    held = open(d).read()
    for text in ("a.o : /elsewhere/pkg/csrc/a.cu /elsewhere/pkg/csrc/one.cuh\n", "a.o :\n", ""):
        write(d, text)
        assert m._stale("a") and m.needs_build()
    write(d, held)
    assert not m._stale("a")
    os.remove(d)
    assert m._stale("a")


def test_a_removed_header_is_seen(built, tmp_path):
    m = tree(built, str(tmp_path / "copy"))
    os.remove(os.path.join(m.CSRC, "one.cuh"))
    assert m._stale("a") and not m._stale("b")


def test_a_failed_compilation_leaves_nothing_behind(built, tmp_path):
    m = tree(built, str(tmp_path / "copy"))
    held = {f: open(os.path.join(m.OBJ, f), "rb").read() for f in os.listdir(m.OBJ)}
    lib = open(m.LIB, "rb").read()
    write(os.path.join(m.CSRC, "a.cu"), "no C\n")
    touch(os.path.join(m.CSRC, "a.cu"))
    touch(os.path.join(m.CSRC, "b.cu"))
    with pytest.raises(subprocess.CalledProcessError):
        m.build()
    assert sorted(os.listdir(m.OBJ)) == sorted(held) and m.needs_build()
    assert [f for f in os.listdir(os.path.dirname(m.LIB)) if "tmp" in f] == [] and open(m.LIB, "rb").read() == lib
    write(os.path.join(m.CSRC, "a.cu"), "extern \"C\" int a() { return 3; }\n")
    m.build()
    assert sorted(os.listdir(m.OBJ)) == sorted(held)
