"""Build libmoe_ffn.so in-tree with nvcc for sm_100a (cross-compiles without a GPU), and _bind.so, the block
operators' binding for torch tensors, with g++."""
import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libmoe_ffn.so")
BIND = os.path.join(HERE, "_bind.so")
BIND_SOURCE = os.path.join(HERE, "csrc", "bind.cpp")
SOURCES = sorted(glob.glob(os.path.join(HERE, "csrc", "*.cu")))
HEADERS = sorted(glob.glob(os.path.join(HERE, "csrc", "*.cuh"))) + [os.path.join(ROOT, "include", "moe_ffn.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr",
    "-Xptxas", "-warn-spills",
]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _older(target, sources) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in sources)


def stale() -> bool:
    return _older(LIB, SOURCES + HEADERS)


def bind_built_for() -> str:
    """What a _bind.so belongs to: it uses torch's C++ interface, which each version changes, and Python's."""
    import torch
    return "torch %s, Python %s" % (torch.__version__, sysconfig.get_config_var("SOABI"))


def bind_stale() -> bool:
    if _older(BIND, [BIND_SOURCE, HEADERS[-1]]):
        return True
    with open(BIND, "rb") as f:  # the module's built_for, which ends with a zero
        return bind_built_for().encode() + b"\0" not in f.read()


def build_bind(force: bool = False, verbose: bool = False) -> str:
    """Compile and link _bind.so against torch and libmoe_ffn.so (found beside it at run time)."""
    if not force and not bind_stale():
        return BIND
    import torch
    tdir = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    tmp = BIND + ".tmp%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, '-DBUILT_FOR="%s"' % bind_built_for()]
    for inc in (os.path.join(tdir, "include"), os.path.join(tdir, "include", "torch", "csrc", "api", "include"),
                os.path.join(cuda, "include"), sysconfig.get_paths()["include"]):
        cmd += ["-isystem", inc]
    cmd += [BIND_SOURCE, "-o", tmp, "-L" + os.path.join(tdir, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_cuda", "-ltorch", "-ltorch_python", "-L" + HERE, "-l:libmoe_ffn.so", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, BIND)
    return BIND


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if force or stale():
        tmp = LIB + ".tmp%d" % os.getpid()
        cmd = [nvcc()] + NVCC_FLAGS + list(extra) + ["-I", os.path.join(ROOT, "include")] + SOURCES + ["-o", tmp]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        subprocess.check_call(cmd)
        os.replace(tmp, LIB)
    build_bind(force=force, verbose=verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
    print(LIB)
