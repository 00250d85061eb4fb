"""Build libdspark.so in-tree for sm_100a with nvcc, and its torch binding with the host compiler.

    python -m speculative_decoding_04_b200.build [--verbose]

The library is written to speculative_decoding_04_b200/lib/libdspark.so, the binding (csrc/binding.cpp)
beside it as an extension module with torch's version in its name: one built against another torch is
never loaded.
"""
import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB_DIR = os.path.join(HERE, "lib")
LIB_PATH = os.path.join(LIB_DIR, "libdspark.so")
BINDING_SRC = os.path.join(HERE, "csrc", "binding.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
    "--expt-relaxed-constexpr",
    "--threads", "0",   # the sources at once
]


def nvcc():
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    p = os.path.join(cuda, "bin", "nvcc")
    return p if os.path.exists(p) else "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.cu")))


def needs_build():
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    deps = sources() + glob.glob(os.path.join(HERE, "csrc", "*.cuh")) + glob.glob(os.path.join(HERE, "csrc", "*.h")) \
        + glob.glob(os.path.join(ROOT, "include", "*.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def run(cmd, what, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, cwd=HERE, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stdout.write(r.stdout)
        sys.stderr.write(r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed building {what}")


def binding_path():
    import torch

    tag = "".join(c if c.isalnum() else "_" for c in torch.__version__)
    return os.path.join(LIB_DIR, f"_binding_torch{tag}" + sysconfig.get_config_var("EXT_SUFFIX"))


def needs_binding():
    path = binding_path()
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(d) > t for d in [BINDING_SRC] + glob.glob(os.path.join(ROOT, "include", "*.h")))


def build_binding(verbose=False):
    import torch

    torch_dir = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    inc = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    path = binding_path()
    tmp = path + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-DTORCH_EXTENSION_NAME=_binding",
           "-DTORCH_API_INCLUDE_EXTENSION_H", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += ["-isystem" + d for d in inc] + [BINDING_SRC, "-o", tmp, "-L" + LIB_DIR, "-l:libdspark.so",
                                            "-L" + os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda",
                                            "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python",
                                            "-Wl,-rpath,$ORIGIN"]
    run(cmd, "the torch binding", verbose)
    os.replace(tmp, path)


def build(verbose=False, force=False, ptxas_verbose=False):
    if force or needs_build():
        build_library(verbose, ptxas_verbose)
    if force or needs_binding():
        build_binding(verbose)
    return LIB_PATH


def build_library(verbose=False, ptxas_verbose=False):
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc()] + NVCC_FLAGS + (["-Xptxas", "-v"] if ptxas_verbose else []) + [
        "-I" + os.path.join(ROOT, "include"), "-shared", "-o", tmp] + sources()
    run(cmd, "libdspark.so", verbose)
    os.replace(tmp, LIB_PATH)


if __name__ == "__main__":
    build(verbose="--verbose" in sys.argv, force=True, ptxas_verbose="--ptxas" in sys.argv)
    print(LIB_PATH)
