"""Build libdfssm.so in-tree for sm_100a (B200) with nvcc.

    python -m bit_scaffold_quantized_b200.build [--force] [--variant phases]

nvcc cross-compiles without a GPU.  The library links the CUDA runtime statically
and exports only the C ABI declared in include/dfssm.h.  The "phases" variant
(libdfssm_phases.so) is the same library with the batch-1 token kernel's per-phase
cycle counters compiled in (-DDFSSM_PHASE_TIMERS), for bit_scaffold_quantized_b200.phases.

Beside the library, g++ builds _binding.so (csrc/binding.cpp): the checks and the marshalling
of PyTorch tensors for the calls that take a few microseconds, against the installed
PyTorch's headers.
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


BINDING = os.path.join(PKG, "_binding.so")
CXX = os.environ.get("CXX", "g++")


def _binding_cmd(out: str):
    """The command that builds csrc/binding.cpp as the extension module _binding."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    cuda = os.path.dirname(os.path.dirname(NVCC))
    inc = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-w", "-DTORCH_EXTENSION_NAME=_binding",
            f"-D_GLIBCXX_USE_CXX11_ABI={abi}", *[a for d in inc for a in ("-isystem", d)], os.path.join(CSRC, "binding.cpp"),
            "-o", out, "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".cpp"))]
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
    if not force and up_to_date(lib) and up_to_date(BINDING):
        return lib
    with tempfile.TemporaryDirectory(prefix="dfssm_build_") as tmp:
        objs = [os.path.join(tmp, src + ".o") for src in SOURCES]
        cmds = [[NVCC, *(["-Xptxas=-v"] if verbose else []), *FLAGS, *defines, "-I", INCLUDE, "-I", CSRC, "-c",
                 os.path.join(CSRC, src), "-o", obj] for src, obj in zip(SOURCES, objs)]
        procs = []
        cmds.append(_binding_cmd(BINDING + ".tmp"))
        for cmd in cmds:                      # the sources compile side by side
            if verbose:
                print(" ".join(cmd))
            procs.append(subprocess.Popen(cmd))
        for cmd, code in zip(cmds, [p.wait() for p in procs]):
            if code:
                raise subprocess.CalledProcessError(code, cmd)
        subprocess.run([NVCC, *FLAGS, "-shared", "-o", lib + ".tmp", *objs], check=True)
    os.replace(lib + ".tmp", lib)
    os.replace(BINDING + ".tmp", BINDING)
    return lib


if __name__ == "__main__":
    v = sys.argv[sys.argv.index("--variant") + 1] if "--variant" in sys.argv else ""
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, variant=v))
