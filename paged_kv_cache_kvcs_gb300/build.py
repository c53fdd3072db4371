"""Build the CUDA library ``_build/libkvcs.so`` for sm_103a with nvcc.

One ``-gencode``; the translation units compile in parallel (the attention
kernels once per cache type) and link into one library, with the CUDA
runtime linked statically so that it needs nothing but the driver at run time.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
OUT_DIR = PKG / "_build"
LIB = OUT_DIR / "libkvcs.so"
# (source, defines) of each object
UNITS = [("kvcs.cu", ()), ("kvcs_attend.cu", ())] + [
    ("kvcs_attend_type.cu", (f"-DKVCS_KV_TYPE={t}",)) for t in range(3)]
DEPS = (sorted(CSRC.glob("*.cu")) + sorted(CSRC.glob("*.cuh")) + sorted(CSRC.glob("*.h"))
        + [INCLUDE / "kvcs.h"])
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not Path(cand).exists():
        raise RuntimeError("nvcc not found: the CUDA toolkit is required")
    return cand


def build(force: bool = False, verbose: bool = False) -> Path:
    """Compile unless the library is newer than every source and header."""
    if (not force and LIB.exists()
            and LIB.stat().st_mtime >= max(p.stat().st_mtime for p in DEPS)):
        return LIB
    OUT_DIR.mkdir(exist_ok=True)
    flags = [ARCH, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
             f"-I{INCLUDE}", f"-I{CSRC}", *(["-Xptxas", "-v"] if verbose else [])]

    tmp = OUT_DIR / f"libkvcs.so.tmp{os.getpid()}"
    with tempfile.TemporaryDirectory(dir=OUT_DIR) as objects_dir:
        def compile_unit(i: int) -> str:
            source, defines = UNITS[i]
            obj = str(Path(objects_dir) / f"unit{i}.o")
            subprocess.run([nvcc(), *flags, *defines, "-c", str(CSRC / source), "-o", obj],
                           check=True)
            return obj

        with ThreadPoolExecutor(len(UNITS)) as ex:
            objects = list(ex.map(compile_unit, range(len(UNITS))))
        subprocess.run([nvcc(), ARCH, "-shared", "-cudart", "static", *objects, "-o", str(tmp)],
                       check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose="-v" in sys.argv))
