"""Build the sm_100a CUDA library libmoe_b200.so and its Python binding in-tree
(next to this file).

    python -m mixture_experts_ffn_token_b200.build [--verbose-ptxas]

nvcc compiles every csrc/*.cu for sm_100a only and links one shared library
exporting the C ABI of include/moe.h (the CUDA runtime is linked statically).
g++ compiles csrc/binding.cpp, which reads torch's tensors, to _binding.so.
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


def up_to_date() -> bool:
    both = [os.path.join(os.path.dirname(HERE), "include", "moe.h"), __file__]
    inputs = {LIB: sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + both, BINDING: [BINDING_SOURCE] + both}
    return all(os.path.exists(out) and all(os.path.getmtime(p) <= os.path.getmtime(out) for p in paths)
               for out, paths in inputs.items())


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
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
    build_binding()
    return LIB


def build_binding():
    import torch
    root = os.path.dirname(torch.__file__)
    include = [sysconfig.get_paths()["include"], os.path.join(root, "include"),
               os.path.join(root, "include", "torch", "csrc", "api", "include"), os.path.join(CUDA_HOME, "include")]
    tmp = f"{BINDING}.{os.getpid()}.tmp"
    subprocess.run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
                    BINDING_SOURCE, "-o", tmp, *(f"-I{d}" for d in include),
                    f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-L" + os.path.join(root, "lib"),
                    "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"], check=True)
    os.replace(tmp, BINDING)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose-ptxas", action="store_true")
    args = ap.parse_args()
    print(build(force=True, verbose_ptxas=args.verbose_ptxas), file=sys.stderr)
