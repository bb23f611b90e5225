"""Build the sm_100a CUDA library libmoe_b200.so and its Python binding in-tree
(next to this file).

    python -m mixture_experts_ffn_token_b200.build [--verbose-ptxas]

nvcc compiles every csrc/*.cu for sm_100a only and links one shared library
exporting the C ABI of include/moe.h (the CUDA runtime is linked statically).
g++ compiles csrc/binding.cpp, which reads torch's tensors, to _binding.so, for
the torch and the Python that run this; without torch only the library is built.
Each of the two is built again when its own inputs have changed.
"""
import argparse
import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmoe_b200.so")
BINDING = os.path.join(HERE, "_binding.so")
BUILD_DIR = os.path.join(HERE, "_build")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
CUDA_HOME = os.environ.get("CUDA_HOME", "/usr/local/cuda")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")


BOTH = [os.path.join(os.path.dirname(HERE), "include", "moe.h"), __file__]


def _newer(out, paths) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(p) <= os.path.getmtime(out) for p in paths)


def binding_target() -> str:
    """What _binding.so is compiled for: it reads these versions' C++ objects."""
    import torch
    return f"torch {torch.__version__}, Python {'.'.join(map(str, sys.version_info[:2]))}, " \
           f"C++11 ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}"


def _target_file() -> str:
    return os.path.join(BUILD_DIR, "binding_target.txt")


def library_up_to_date() -> bool:
    return _newer(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + BOTH)


def binding_up_to_date() -> bool:
    if not _newer(BINDING, [BINDING_SOURCE] + BOTH) or not os.path.exists(_target_file()):
        return False
    with open(_target_file()) as f:
        return f.read() == binding_target()


def up_to_date() -> bool:
    return library_up_to_date() and binding_up_to_date()


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    if force or not library_up_to_date():
        build_library(verbose_ptxas)
    try:
        import torch  # noqa: F401
    except ImportError as e:
        print(f"_binding.so is not built: it needs torch ({e})", file=sys.stderr)
    else:
        if force or not binding_up_to_date():
            build_binding()
    return LIB


def build_library(verbose_ptxas: bool = False):
    objs = []
    for src in sources():
        obj = os.path.join(BUILD_DIR, os.path.basename(src).replace(".cu", ".o"))
        cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
        if verbose_ptxas:
            cmd += ["-Xptxas", "-v"]
        subprocess.run(cmd, check=True)
        objs.append(obj)
    tmp = LIB + ".tmp"
    subprocess.run([NVCC, *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs, "-o", tmp], check=True)
    os.replace(tmp, LIB)


def build_binding():
    import torch
    root = os.path.dirname(torch.__file__)
    include = [sysconfig.get_paths()["include"], os.path.join(root, "include"),
               os.path.join(root, "include", "torch", "csrc", "api", "include"), os.path.join(CUDA_HOME, "include")]
    tmp = f"{BINDING}.{os.getpid()}.tmp"
    subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
                    BINDING_SOURCE, "-o", tmp, *(f"-I{d}" for d in include),
                    f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                    f'-DMOE_BINDING_TARGET="{binding_target()}"', "-L" + os.path.join(root, "lib"),
                    "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"], check=True)
    os.replace(tmp, BINDING)
    with open(_target_file(), "w") as f:
        f.write(binding_target())


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose-ptxas", action="store_true")
    args = ap.parse_args()
    print(build(force=True, verbose_ptxas=args.verbose_ptxas), file=sys.stderr)
