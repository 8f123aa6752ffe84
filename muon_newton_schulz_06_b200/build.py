"""Builds the sm_100a shared library libmuon_b200.so next to this file.

    python -m muon_newton_schulz_06_b200.build [--verbose-ptxas]

nvcc compiles every kernel for sm_100a only (tcgen05 / TMA / TMEM instructions) and
links the CUDA runtime statically, so the library needs no libcudart at load time.
g++ compiles the binding's marshalling module _muon_py (CPython C API) for the interpreter
that runs the build; its file name carries that interpreter's tag.
"""
import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libmuon_b200.so")
PY_SOURCE = os.path.join(HERE, "csrc", "muon_py.cpp")
PY_LIB = os.path.join(HERE, "_muon_py" + sysconfig.get_config_var("EXT_SUFFIX"))
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def sources():
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.cu")))


def up_to_date():
    if not os.path.exists(LIB) or not os.path.exists(PY_LIB):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(PY_LIB))
    deps = (sources() + [PY_SOURCE] + glob.glob(os.path.join(HERE, "csrc", "*.h")) + glob.glob(os.path.join(HERE, "csrc", "*.cuh"))
            + glob.glob(os.path.join(ROOT, "include", "*.h")))
    return all(os.path.getmtime(d) <= t for d in deps)


def build(verbose_ptxas=False, force=False):
    if not force and up_to_date():
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    cmd = [nvcc, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-shared", "-Xcompiler", "-fPIC",
           "-Xcompiler", "-fvisibility=hidden", "-cudart", "static", "--threads", "0",
           "-I", os.path.join(ROOT, "include"), "-o", LIB + ".tmp", *sources()]
    if verbose_ptxas:
        cmd[1:1] = ["-Xptxas", "-v"]
    subprocess.run(cmd, check=True)
    os.replace(LIB + ".tmp", LIB)
    subprocess.run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
                    "-I", os.path.join(ROOT, "include"), "-I", sysconfig.get_paths()["include"],
                    "-o", PY_LIB + ".tmp", PY_SOURCE], check=True)
    os.replace(PY_LIB + ".tmp", PY_LIB)
    untagged = os.path.join(HERE, "_muon_py.so")      # of an earlier build: any interpreter would take it
    if os.path.exists(untagged):
        os.remove(untagged)
    return LIB


if __name__ == "__main__":
    build(verbose_ptxas="--verbose-ptxas" in sys.argv, force=True)
    print(LIB)
