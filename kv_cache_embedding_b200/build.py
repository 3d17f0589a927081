"""Build libtq.so (the sm_100a CUDA library behind include/tq.h) and _kv8.so (the
torch side of its paged-cache calls) in-tree."""
import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libtq.so")
BIND_SRC = os.path.join(CSRC, "kv8_bind.cpp")
BIND = os.path.join(PKG, "_kv8.so")

NVCC_FLAGS = [
    "-std=c++17", "-O3", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _older(path, deps):
    return not os.path.exists(path) or any(os.path.getmtime(p) > os.path.getmtime(path) for p in deps)


def _stale_lib():
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    return _older(LIB, deps + [os.path.join(INCLUDE, "tq.h")])


def _torch_version():
    from importlib.metadata import version
    return version("torch")


def _stale_bind():
    """_kv8.so is older than its sources, or built for another torch (whose C++
    interface it is bound to)."""
    deps = [BIND_SRC] + glob.glob(os.path.join(CSRC, "*.h")) + [os.path.join(INCLUDE, "tq.h")]
    if _older(BIND, deps):
        return True
    with open(BIND, "rb") as f:
        return b"built for torch " + _torch_version().encode() + b"\0" not in f.read()


def _stale():
    return _stale_lib() or _stale_bind()


def _bind_command(out):
    """g++ over kv8_bind.cpp against this interpreter's torch."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    inc = [INCLUDE, os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    return ["g++", "-std=c++17", "-O2", "-shared", "-fPIC", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            f"-DTQ_TORCH={_torch_version()}",
            *(f"-I{i}" for i in inc), BIND_SRC, "-o", out,
            f"-L{PKG}", "-l:libtq.so", "-Wl,-rpath,$ORIGIN", f"-L{os.path.join(root, 'lib')}",
            "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]


def build(force=False, verbose=False):
    """Compile every .cu under csrc/ for sm_100a and link libtq.so (static
    CUDA runtime; the driver API is reached through cudaGetDriverEntryPoint);
    then _kv8.so."""
    if force or _stale_lib():
        _build_lib(verbose)
    if force or _stale_bind():
        subprocess.check_call(_bind_command(BIND + ".tmp"))
        os.replace(BIND + ".tmp", BIND)
    return LIB


def _build_lib(verbose):
    nvcc = os.environ.get("NVCC", "nvcc")
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    procs = []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [nvcc, *NVCC_FLAGS, "-I", INCLUDE, "-dc" if False else "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd))
        procs.append((subprocess.Popen(cmd), src))
        objs.append(obj)
    for p, src in procs:
        if p.wait() != 0:
            raise RuntimeError(f"nvcc failed on {src}")
    tmp = LIB + ".tmp"
    cmd = [nvcc, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-o", tmp, *objs]
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
