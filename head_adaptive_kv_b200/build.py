"""Build ``libhkv.so`` (the sm_100a CUDA library behind ``include/*.h``) in-tree:
one object per source, compiled side by side, then one link."""
import glob
import os
import re
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libhkv.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs(path, seen=None):
    """A source and the files of this repository that it includes."""
    seen = set() if seen is None else seen
    if path in seen:
        return seen
    seen.add(path)
    with open(path) as f:
        for name in re.findall(r'^\s*#include "([^"]+)"', f.read(), flags=re.M):
            for folder in (CSRC, INCLUDE):
                if os.path.exists(os.path.join(folder, name)):
                    _inputs(os.path.join(folder, name), seen)
    return seen


def _newest(paths) -> float:
    return max(os.path.getmtime(p) for p in paths)


def _object(src):
    return os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")


def build(force: bool = False, verbose: bool = False) -> str:
    need = {src: _newest(_inputs(src)) for src in sources()}
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= max(need.values()):
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    os.makedirs(OBJ, exist_ok=True)

    def compile_one(src):
        obj = _object(src)
        if not force and os.path.exists(obj) and os.path.getmtime(obj) >= need[src]:
            return
        subprocess.run([nvcc, *NVCC_FLAGS, "-I", INCLUDE, *(["-Xptxas", "-v"] if verbose else []), "-c", src,
                        "-o", obj + ".tmp"], check=True)
        os.replace(obj + ".tmp", obj)

    with ThreadPoolExecutor(max_workers=len(need)) as pool:
        list(pool.map(compile_one, need))
    subprocess.run([nvcc, *NVCC_FLAGS, "-shared", *map(_object, need), "-o", LIB + ".tmp"], check=True)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
