"""Build libpasa.so in-tree with nvcc for sm_103a: one object for each csrc/*.cu, side by side, then
linked. An object is made again when its source, or a header it included, is newer."""
from __future__ import annotations

import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpasa.so")
NVCC_FLAGS = [
    "-std=c++17", "-O3", "-lineinfo",
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-Xcompiler", "-fPIC",
]


def _units():
    return sorted(f[:-3] for f in os.listdir(CSRC) if f.endswith(".cu"))


def _newer(target: str, sources) -> bool:
    """Whether target is missing or older than one of its sources (a missing source counts as new)."""
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(not os.path.exists(s) or os.path.getmtime(s) > t for s in sources)


def _depends(unit: str):
    """What the object of a unit was made from: this file, and the sources its dependency file lists, by their places relative to
    csrc/, which a copied or moved tree keeps. Without the unit's own source there (no list, or one of another
    kind) the object counts as old; the toolkit's headers, which have absolute paths, are not looked at."""
    own = os.path.join(CSRC, unit + ".cu")
    try:
        with open(os.path.join(OBJ, unit + ".d")) as f:
            listed = f.read().replace("\\\n", " ").partition(":")[2].split()
    except OSError:
        listed = []
    sources = [os.path.normpath(os.path.join(CSRC, s)) for s in listed if not os.path.isabs(s)]
    return [os.path.abspath(__file__), own] + (sources if own in sources else [own + ".missing"])


def _stale(unit: str) -> bool:
    return _newer(os.path.join(OBJ, unit + ".o"), _depends(unit))


def needs_build() -> bool:
    return any(_stale(u) for u in _units()) or _newer(LIB, [os.path.join(OBJ, u + ".o") for u in _units()])


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the units that changed and link libpasa.so next to this file; returns its path."""
    if not force and not needs_build():
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    os.makedirs(OBJ, exist_ok=True)
    tag = f".tmp{os.getpid()}"
    made = []   # under their final names

    def place(path):
        made.append(path)
        return path + tag

    try:
        running = []
        for unit in _units():
            if force or _stale(unit):
                # in csrc/ and with relative paths, so that the dependency file holds relative ones
                cmd = [nvcc, *NVCC_FLAGS, "-c", "-MMD", "-MF", place(os.path.join(OBJ, unit + ".d")), "-o",
                       place(os.path.join(OBJ, unit + ".o")), unit + ".cu"]
                if verbose:
                    cmd.insert(1, "-Xptxas=-v")
                running.append(subprocess.Popen(cmd, cwd=CSRC))
        failed = [p.args for p in running if p.wait() != 0]   # all of them end before one is reported
        if failed:
            raise subprocess.CalledProcessError(1, failed[0])
        for path in made:
            os.replace(path + tag, path)
        subprocess.run([nvcc, "-shared", "-gencode", "arch=compute_103a,code=sm_103a", "-o", place(LIB),
                        *(os.path.join(OBJ, u + ".o") for u in _units())], check=True)
        os.replace(LIB + tag, LIB)
    finally:
        for path in made:
            if os.path.exists(path + tag):
                os.remove(path + tag)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
