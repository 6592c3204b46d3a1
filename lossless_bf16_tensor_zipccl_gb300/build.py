"""Build libzipccl.so (the sm_103a kernels and the C ABI) in-tree with nvcc,
and the extension that makes the operator calls on torch tensors with g++.

Translation units compile in parallel; the shared library lands in
``lossless_bf16_tensor_zipccl_gb300/_build/libzipccl.so``, the extension beside
it under a name that holds the Python and torch versions it was built for.
"""
from __future__ import annotations

import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libzipccl.so")
SOURCES = ["zc_api.cu", "zc_encode.cu", "zc_decode.cu", "zc_noalloc.cu", "zc_codebook.cpp", "zc_route.cu",
           "zc_dispatch.cu", "zc_adamw.cu", "zc_quantize.cu", "zc_matmul.cu", "zc_layer_up.cu",
           "zc_layer_down.cu"]
HEADERS = ["zc_format.h", "zc_device.cuh", "zc_kernels.h", "zc_codebook.h", "zc_ops.cuh", "zc_fp8.cuh",
           "zc_tensor.cuh", "zc_route.cuh", "zc_layer.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
# No fast-math: the reduce folds in IEEE fp32 with subnormals kept.
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-ftz=false", "-prec-div=true",
              "-prec-sqrt=true", "-fmad=false", "-I" + os.path.join(HERE, "..", "include")]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libzipccl")
    return cand


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(HERE, "..", "include", "zipccl.h"),
                                                                 os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        if verbose or ptxas_info:
            print(r.stderr, end="")
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


def torch_extension(force: bool = False) -> str:
    """Path of the torch extension, built with g++ when missing or stale."""
    import sysconfig

    import torch
    tag = f"{sysconfig.get_config_var('SOABI')}-torch{torch.__version__}"
    out = os.path.join(BUILD, f"_zipccl_torch.{tag}.so")
    src = os.path.join(CSRC, "zc_torch.cpp")
    header = os.path.join(HERE, "..", "include", "zipccl.h")
    if not force and os.path.exists(out) and all(os.path.getmtime(d) <= os.path.getmtime(out)
                                                 for d in (src, header, os.path.abspath(__file__))):
        return out
    build()
    root = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"), cuda,
               sysconfig.get_paths()["include"], os.path.dirname(header)]
    tmp = out + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *("-I" + i for i in include), src, "-o", tmp, "-L" + BUILD, "-lzipccl", "-Wl,-rpath,$ORIGIN",
           "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-ltorch_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on zc_torch.cpp:\n{r.stderr}")
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
    print(torch_extension(force="--force" in sys.argv))
