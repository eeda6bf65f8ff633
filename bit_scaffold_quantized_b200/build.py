"""Build libdfssm.so in-tree for sm_100a (B200) with nvcc.

    python -m bit_scaffold_quantized_b200.build [--force] [--variant phases]

nvcc cross-compiles without a GPU.  The library links the CUDA runtime statically
and exports only the C ABI declared in include/dfssm.h.  The "phases" variant
(libdfssm_phases.so) is the same library with the batch-1 token kernel's per-phase
cycle counters compiled in (-DDFSSM_PHASE_TIMERS), for bit_scaffold_quantized_b200.phases.
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libdfssm.so")
VARIANTS = {"": ([], LIB), "phases": (["-DDFSSM_PHASE_TIMERS"], os.path.join(PKG, "libdfssm_phases.so"))}
SOURCES = ["dfssm_api.cu", "mixer_api.cu"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-fvisibility=hidden",
    "-cudart", "static",
    "--expt-relaxed-constexpr",
]


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))]
    files.append(os.path.join(INCLUDE, "dfssm.h"))
    files.append(os.path.abspath(__file__))
    return files


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False, variant: str = "") -> str:
    defines, lib = VARIANTS[variant]
    if not force and up_to_date(lib):
        return lib
    with tempfile.TemporaryDirectory(prefix="dfssm_build_") as tmp:
        objs = [os.path.join(tmp, src + ".o") for src in SOURCES]
        cmds = [[NVCC, *(["-Xptxas=-v"] if verbose else []), *FLAGS, *defines, "-I", INCLUDE, "-I", CSRC, "-c",
                 os.path.join(CSRC, src), "-o", obj] for src, obj in zip(SOURCES, objs)]
        procs = []
        for cmd in cmds:                      # the sources compile side by side
            if verbose:
                print(" ".join(cmd))
            procs.append(subprocess.Popen(cmd))
        for cmd, code in zip(cmds, [p.wait() for p in procs]):
            if code:
                raise subprocess.CalledProcessError(code, cmd)
        subprocess.run([NVCC, *FLAGS, "-shared", "-o", lib + ".tmp", *objs], check=True)
    os.replace(lib + ".tmp", lib)
    return lib


if __name__ == "__main__":
    v = sys.argv[sys.argv.index("--variant") + 1] if "--variant" in sys.argv else ""
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, variant=v))
