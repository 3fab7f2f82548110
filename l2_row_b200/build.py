"""Build libds.so (the CUDA library) in-tree for sm_100a.

    python -m l2_row_b200.build [--force]

nvcc cross-compiles without a GPU.  The shared library lands next to this
file so it travels with the source tree; the Python binding loads it from
there and nowhere else.
"""
from __future__ import annotations

import contextlib
import hashlib
import mmap
import os
import re
import shutil
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libds.so")
SOURCES = ["ds_kernels.cu", "ds_tile.cu", "ds_qk.cu", "ds_col.cu", "ds_embed.cu", "ds_qkn.cu", "ds_logp.cu", "ds_api.cpp", "ds_lm_api.cpp"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2,-Wall",
    "-Xptxas", "-warn-spills",
]
LINK_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-Xlinker", "-z,defs"]  # no name undefined
LINK_LIBS = ["-lcudart_static", "-lrt", "-lpthread", "-ldl"]


def nvcc() -> str | None:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    return None


def _digest(*parts) -> str:
    h = hashlib.sha256()
    for p in parts:
        b = p if isinstance(p, bytes) else str(p).encode()
        h.update(b"%d:" % len(b) + b)
    return h.hexdigest()


def _read(path: str) -> bytes:
    with open(path, "rb") as f:
        return f.read()


def _files_of(path: str) -> list[str]:
    """The source and every header of this project that it includes, at any depth."""
    todo, found = [path], []
    while todo:
        p = todo.pop()
        if p in found:
            continue
        found.append(p)
        for name in re.findall(rb'^\s*#\s*include\s*"([^"]+)"', _read(p), re.M):
            for d in (os.path.dirname(p), CSRC, INCLUDE):
                q = os.path.normpath(os.path.join(d, name.decode()))
                if os.path.exists(q):
                    todo.append(q)
                    break
    return found


def source_key(src: str) -> str:
    """What an object depends on besides the compiler: the text of its source
    and headers and the flags.  File times say nothing: a copy does not keep
    them, and a failed compilation leaves an older object behind."""
    texts = [(os.path.basename(p), _read(p)) for p in sorted(_files_of(os.path.join(CSRC, src)))]
    return _digest(" ".join(NVCC_FLAGS), src, *(x for t in texts for x in t))


def sources_key() -> str:
    """What the library depends on besides the compiler."""
    return _digest(*(source_key(s) for s in SOURCES), " ".join(LINK_FLAGS + LINK_LIBS))


def library_keys(lib: str) -> tuple[str, str] | None:
    """(sources_key, digest of the compiler's version) that a library was built with."""
    if not os.path.exists(lib) or not os.path.getsize(lib):
        return None
    with open(lib, "rb") as f, mmap.mmap(f.fileno(), 0, access=mmap.ACCESS_READ) as text:
        m = re.search(rb"libds of sources ([0-9a-f]{64}) by compiler ([0-9a-f]{64})", text)
        return (m[1].decode(), m[2].decode()) if m else None


def build(force: bool = False, verbose: bool = False) -> str:
    """Bring libds.so up to date with its sources and the compiler; return its
    path.  An object's file is named after what it was made of (source_key and
    the compiler), so one made of anything else is never linked."""
    cc, have, sources = nvcc(), library_keys(LIB), sources_key()
    if cc is None:
        if have and have[0] == sources and not force:
            return LIB
        raise RuntimeError("nvcc not found: libds.so cannot be built")
    version = _digest(subprocess.run([cc, "--version"], capture_output=True, check=True).stdout)
    keys = (sources, version)
    if not force and have == keys:
        return LIB
    tmpdir = os.path.join(HERE, "_build")
    os.makedirs(tmpdir, exist_ok=True)
    objs = []
    # what is being written has a folder of its own: an object or a library
    # takes its place whole, or, where its compiler failed, not at all
    with tempfile.TemporaryDirectory(dir=tmpdir) as new:
        procs = []
        for src in SOURCES:
            obj = os.path.join(tmpdir, f"{src}.{_digest(source_key(src), version)[:32]}.o")
            objs.append(obj)
            if not force and os.path.exists(obj):
                continue
            cmd = [cc, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o",
                   os.path.join(new, src + ".o")]
            if verbose:
                print(" ".join(cmd))
            procs.append((src, subprocess.Popen(cmd), obj))
        failed = []
        for src, p, obj in procs:  # every compiler ends before this call does
            if p.wait() == 0:
                os.replace(os.path.join(new, src + ".o"), obj)
            else:
                failed.append(src)
        if failed:
            raise RuntimeError(f"nvcc failed building libds.so: {', '.join(failed)}")
        key, lib = os.path.join(new, "key.cpp"), os.path.join(new, "libds.so")
        with open(key, "w") as f:
            f.write(f'extern "C" const char ds_build_key[] = "libds of sources {keys[0]} by compiler {keys[1]}";\n')
        subprocess.run([cc, *NVCC_FLAGS, "-c", key, "-o", key + ".o"], check=True)
        subprocess.run([cc, *LINK_FLAGS, "-o", lib, *objs, key + ".o", *LINK_LIBS], check=True)
        os.replace(lib, LIB)
    for name in os.listdir(tmpdir):  # objects of earlier texts
        path = os.path.join(tmpdir, name)
        if os.path.isfile(path) and path not in objs:
            with contextlib.suppress(FileNotFoundError):  # another build's removal
                os.remove(path)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
