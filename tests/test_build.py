"""Building the library (no GPU): the sources compile, what is built is what
the binding loads, and nothing that was made of other sources takes its place
(with a compiler that only copies its input)."""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys

import pytest

from l2_row_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_sources_build_and_the_binding_loads():
    """Every source compiles (at once where the library is up to date), and
    every name that the binding declares is in the library."""
    assert build.build() == build.LIB
    code = "from l2_row_b200 import ds; assert all(hasattr(ds.lib(), n) for n in ds.EXPORTS)"
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True)


# An "object" is its source's text with the headers it names, the "library" all
# objects; a source that holds BROKEN does not compile.
COPYING_COMPILER = """#!/bin/sh
out= src= objs=
while [ $# -gt 0 ]; do
    case $1 in
    --version) echo copying; exit 0;;
    -o) out=$2; shift;;
    -c) src=$2; shift;;
    *.o) objs="$objs $1";;
    esac
    shift
done
[ -z "$src" ] && exec cat $objs > "$out"
echo "$src" >> "$LOG"
echo half > "$out"
grep -q SLOW "$src" && sleep 1
grep -q BROKEN "$src" && exit 1
dir=$(dirname "$src")
cat "$src" $(sed -n 's/^#include "\\(ds_[a-z_]*\\.cuh\\{0,1\\}\\)"/\\1/p' "$src" | sed "s|^|$dir/|") > "$out"
[ -z "$LOG" ] || echo "done $src" >> "$LOG"
"""


class Tree:
    """A copy of the package's sources and build module under `root`."""

    def __init__(self, root):
        self.root = str(root)
        spec = importlib.util.spec_from_file_location("tree_build", os.path.join(self.root, "l2_row_b200", "build.py"))
        self.build = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(self.build)

    @classmethod
    def copy(cls, root, of=ROOT):
        for d in ("include", "l2_row_b200"):
            shutil.copytree(os.path.join(of, d), os.path.join(root, d), copy_function=shutil.copy,
                            ignore=shutil.ignore_patterns("_build", "*.so", "__pycache__") if of == ROOT else None)
        return cls(root)

    def path(self, name):
        return os.path.join(self.root, "l2_row_b200", "csrc", name)

    def edit(self, name, text):
        with open(self.path(name), "a") as f:
            f.write(text)

    def library(self):
        with open(os.path.join(self.root, "l2_row_b200", "libds.so")) as f:
            return f.read()

    def times(self, when):
        """Every file of the sources dated `when`."""
        for d, _, names in os.walk(self.root):
            for n in names:
                if "_build" not in d and not n.endswith(".so"):
                    os.utime(os.path.join(d, n), (when, when))


@pytest.fixture
def tree(tmp_path, monkeypatch):
    cc = tmp_path / "nvcc"
    cc.write_text(COPYING_COMPILER)
    cc.chmod(0o755)
    monkeypatch.setenv("NVCC", str(cc))
    monkeypatch.setenv("LOG", str(tmp_path / "log"))
    t = Tree.copy(str(tmp_path / "tree"))
    t.build.build()
    return t


def test_objects_of_other_text_are_not_linked(tree, tmp_path):
    """Whatever the files' times say: sources dated before the objects and the
    library, a header, a tree copied elsewhere with its objects."""
    old = os.path.getmtime(os.path.join(tree.root, "l2_row_b200", "libds.so")) - 1000
    tree.edit("ds_qkn.cu", "\n// first edit\n")
    tree.times(old)
    tree.build.build()
    assert tree.library().count("first edit") == 1
    tree.edit("ds_lm.cuh", "\n// header edit\n")
    tree.times(old)
    tree.build.build()
    assert tree.library().count("header edit") == 3         # ds_embed.cu, ds_qkn.cu, ds_logp.cu
    other = Tree.copy(str(tmp_path / "other"), of=tree.root)
    other.edit("ds_lm.h", "\n// third edit\n")
    other.edit("ds_logp.cu", "\n// fourth edit\n")
    other.times(old)
    other.build.build()
    lib = other.library()
    assert lib.count("fourth edit") == 1 and lib.count("first edit") == 1
    assert "fourth edit" not in tree.library()


def test_only_what_changed_is_compiled(tree, tmp_path):
    log = tmp_path / "log"
    log.write_text("")
    assert tree.build.build() and log.read_text() == ""
    tree.edit("ds_qk.cu", "\n// edit\n")
    tree.build.build()
    built = {os.path.basename(x) for x in log.read_text().split("\n") if x and not x.startswith("done")}
    assert built == {"ds_qk.cu", "key.cpp"}        # key.cpp: the library's digest


def test_a_current_library_needs_no_compiler(tree, monkeypatch):
    monkeypatch.setattr(tree.build, "nvcc", lambda: None)
    assert tree.build.build() == os.path.join(tree.root, "l2_row_b200", "libds.so")
    tree.edit("ds_qk.cu", "\n// edit\n")
    with pytest.raises(RuntimeError, match="nvcc not found"):
        tree.build.build()


def test_a_failed_build_leaves_everything_as_it_was(tree, tmp_path):
    """The old library stays, the call ends after every compiler has, no object
    of a failed compilation is left, and the next build makes what is missing."""
    before, log = tree.library(), tmp_path / "log"
    tree.edit("ds_api.cpp", "\nBROKEN\n")
    tree.edit("ds_tile.cu", "\n// SLOW\n")
    log.write_text("")
    with pytest.raises(RuntimeError, match="ds_api.cpp"):
        tree.build.build()
    assert tree.library() == before
    ended = {os.path.basename(x.split()[1]) for x in log.read_text().split("\n") if x.startswith("done")}
    assert ended == {"ds_tile.cu"}
    objects = os.path.join(tree.root, "l2_row_b200", "_build")
    assert sorted(n.split(".")[0] + n[-2:] for n in os.listdir(objects) if n.startswith("ds_api")) == ["ds_api.o"]
    assert not any(os.path.isdir(os.path.join(objects, n)) for n in os.listdir(objects))
    with open(tree.path("ds_api.cpp")) as f:
        text = f.read()
    with open(tree.path("ds_api.cpp"), "w") as f:
        f.write(text.replace("BROKEN", "// mended"))
    tree.build.build()
    assert tree.library().count("// mended") == 1 and tree.library().count("// SLOW") == 1
    assert "half" not in tree.library().split("\n")


@pytest.mark.skipif(build.nvcc() is None, reason="needs nvcc")
def test_an_undefined_name_is_an_error_of_the_build(tmp_path):
    """Not of the program that loads the library."""
    t = Tree.copy(str(tmp_path / "tree"))
    t.build.SOURCES = ["caller.cpp"]
    with open(t.path("caller.cpp"), "w") as f:
        f.write('int not_there(int);\nextern "C" int ds_version(void) { return not_there(1); }\n')
    with pytest.raises(subprocess.CalledProcessError):
        t.build.build()
    assert not os.path.exists(t.build.LIB)
    t.edit("caller.cpp", "int not_there(int i) { return i; }\n")
    assert os.path.exists(t.build.build())


def test_the_binding_refuses_a_library_of_other_sources(tmp_path):
    t = Tree.copy(str(tmp_path / "tree"))
    os.symlink(build.LIB, t.build.LIB)

    def load():
        return subprocess.run([sys.executable, "-c", "import l2_row_b200.ds"], cwd=t.root, capture_output=True, text=True)

    assert load().returncode == 0
    t.edit("ds_lm.h", "\n// another layout\n")
    r = load()
    assert r.returncode != 0 and "not built from the sources beside it" in r.stderr
    shutil.rmtree(os.path.join(t.root, "l2_row_b200", "csrc"))     # a package without sources
    assert load().returncode == 0


def test_builds_at_once(tree):
    """Processes that build one tree together all succeed, on the same library."""
    tree.edit("ds_tile.cu", "\n// SLOW together\n")
    code = "from l2_row_b200 import build; build.build()"
    for edit in range(3):
        tree.edit("ds_lm.h", f"\n// edit {edit}\n")
        procs = [subprocess.Popen([sys.executable, "-c", code], cwd=tree.root, stderr=subprocess.PIPE) for _ in range(6)]
        ends = [(p.communicate()[1], p.returncode) for p in procs]
        assert all(rc == 0 for _, rc in ends), ends
        assert tree.build.library_keys(tree.build.LIB)[0] == tree.build.sources_key()
    assert tree.library().count("SLOW together") == 1
