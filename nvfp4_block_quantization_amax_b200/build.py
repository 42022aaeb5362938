"""Build libnvfp4.so in-tree with nvcc for sm_100a, and _fastcall.*.so, the C++
host path of the small calls, with the host compiler against torch's headers.

The library is plain CUDA C++ behind the C ABI of include/nvfp4.h.  Every
translation unit is compiled with -fmad=false so no multiply-add is fused:
the quantizer's arithmetic is one rounding per operation, like its CPU
restatement.
"""
import glob
import os
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libnvfp4.so")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo", "-fmad=false",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale():
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) \
        + [os.path.join(INCLUDE, "nvfp4.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def fastcall_path():
    """The small calls' host path for this torch and this Python, whose layouts
    are compiled into it: its name says which, so that no other one's is taken."""
    import torch
    return os.path.join(PKG, f"_fastcall.torch-{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")


def build_fastcall(force=False, verbose=False):
    out = fastcall_path()
    src = os.path.join(CSRC, "fastcall.cpp")
    deps = (src, os.path.join(INCLUDE, "nvfp4.h"))
    if not force and os.path.exists(out) and all(os.path.getmtime(d) <= os.path.getmtime(out) for d in deps):
        return out
    import torch
    from torch.utils.cpp_extension import include_paths, library_paths
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    headers = [*include_paths(), os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I", INCLUDE,
           *(f for h in headers for f in ("-isystem", h)), src, "-o", out + ".tmp",
           *(f"-L{d}" for d in library_paths()), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(out + ".tmp", out)
    return out


def build(force=False, verbose=False, extra=()):
    """The library, which needs nvcc alone; then the small calls' host path,
    which needs torch and its headers, and is left out with a warning where it
    cannot be built."""
    _build_library(force, verbose, extra)
    try:
        build_fastcall(force, verbose)
    except (ImportError, OSError, subprocess.CalledProcessError) as e:
        warnings.warn(f"_fastcall, the small calls' host path, was not built: {e}", RuntimeWarning, stacklevel=2)
    return LIB


def _build_library(force, verbose, extra):
    if not force and not _stale():
        return
    nvcc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    objs = []
    outdir = os.path.join(PKG, "_build")
    os.makedirs(outdir, exist_ok=True)
    for src in sources():
        obj = os.path.join(outdir, os.path.basename(src) + ".o")
        cmd = [nvcc, *NVCC_FLAGS, *extra, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)
        objs.append(obj)
    tmp = LIB + ".tmp"
    subprocess.run([nvcc, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", *objs, "-o", tmp],
                   check=True)
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
