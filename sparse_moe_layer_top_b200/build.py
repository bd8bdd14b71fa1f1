"""Build libmoe.so (sm_100a) in-tree with nvcc, and the C++ side of the Python
binding, _moe_binding, with g++.

    python -m sparse_moe_layer_top_b200.build [--force] [--verbose-ptxas] [--checks]

--checks builds the bounds-checking variant libmoe_checks.so instead
(-DMOE_CHECKS: device checks of the kernels' computed and read indices,
reported through the device status word); the binding loads it when the
environment sets MOE_CHECKS=1.
"""
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmoe.so")
LIB_CHECKS = os.path.join(HERE, "libmoe_checks.so")
BINDING = os.path.join(HERE, "_moe_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
SOURCES = [os.path.join(CSRC, "api.cu")]
DEPS = ([os.path.join(CSRC, f) for f in os.listdir(CSRC) if not f.endswith(".cpp")] +
        [os.path.join(ROOT, "include", "moe.h")])
BINDING_DEPS = [BINDING_SOURCE, os.path.join(ROOT, "include", "moe.h")]

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++20", "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC,-O2,-fvisibility=hidden",
    "-shared", "-cudart", "static",
]


def stale(lib=LIB, deps=DEPS):
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(f) > t for f in deps if os.path.isfile(f))


def build_binding(force=False):
    """The binding's C++ side, against this interpreter and its torch."""
    if not force and not stale(BINDING, BINDING_DEPS):
        return BINDING
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")
    tmp = BINDING + ".tmp.%d" % os.getpid()
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
                    "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
                    "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
                    "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda, BINDING_SOURCE, "-o", tmp,
                    "-L" + libs, "-Wl,-rpath," + libs, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"],
                   check=True)
    os.replace(tmp, BINDING)
    return BINDING


def build(force=False, ptxas_verbose=False, checks=False):
    lib = LIB_CHECKS if checks else LIB
    if not force and not stale(lib):
        return lib
    tmp = lib + ".tmp.%d" % os.getpid()
    cmd = ([NVCC] + FLAGS + (["-DMOE_CHECKS"] if checks else []) + (["-Xptxas", "-v"] if ptxas_verbose else []) +
           ["-o", tmp] + SOURCES)
    subprocess.run(cmd, check=True)
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, ptxas_verbose="--verbose-ptxas" in sys.argv,
                checks="--checks" in sys.argv))
    if "--checks" not in sys.argv:
        print(build_binding(force="--force" in sys.argv))
