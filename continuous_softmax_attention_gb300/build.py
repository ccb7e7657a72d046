"""Builds libcsa.so in-tree with nvcc for sm_103a, and the CPython module
_csa_torch (csrc/csa_torch.cpp) that calls it on torch tensors.

Nineteen translation units compiled in parallel, then linked into one shared
library next to this file; the module is compiled beside them against torch's
headers and linked against that library, or left out where torch was built
without CUDA (the library and its ctypes binding do not need it).  The CUDA runtime is linked statically; the CUDA
driver is reached at run time through the runtime's driver entry points, so
the library loads on a machine without a GPU driver (calls then fail with
CSA_ERR_NO_DEVICE).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(HERE, "libcsa.so")
SOURCES = ["csa_api.cu", "csa_simt.cu", "csa_tc.cu", "csa_tc_std.cu", "csa_decode.cu",
           "csa_bwd_simt.cu", "csa_tc_bwd.cu", "csa_host.cu", "csa_noalloc.cu", "csa_paged.cu",
           "csa_rope.cu", "csa_cache.cu", "csa_quant.cu", "csa_paged_e4m3.cu", "csa_paged_int8.cu",
           "csa_tree.cu", "csa_rows_bf16.cu", "csa_rows_e4m3.cu", "csa_rows_int8.cu"]
TORCH_SOURCE = "csa_torch.cpp"
TORCH_LIB_PATH = os.path.join(HERE, "_csa_torch.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc():
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return cand


def nvcc_flags(extra=()):
    return ARCH + [
        "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
        "-I", INCLUDE, "-I", CSRC,
    ] + list(extra)


def build(verbose: bool = False, extra_flags=()) -> str:
    nvcc = _nvcc()
    build_dir = os.path.join(ROOT, "_build")
    os.makedirs(build_dir, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(build_dir, src.replace(".cu", ".o"))
        cmd = [nvcc] + nvcc_flags(extra_flags) + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
        if verbose and (res.stdout or res.stderr):
            print(res.stdout + res.stderr, flush=True)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        module = ex.submit(compile_module, build_dir, verbose) if torch_has_cuda() else None
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcudart_static", "-ldl", "-lpthread", "-lrt"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB_PATH)
    if module is None:
        print("torch has no CUDA half: _csa_torch is left out, its calls raise", file=sys.stderr)
    else:  # behind the library, which does not need it
        link_module(module.result(), verbose)
    return LIB_PATH


def _run(cmd, verbose, what):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{res.stdout}\n{res.stderr}")


def torch_has_cuda():
    """Whether torch brings the headers and libraries that the module needs."""
    import torch

    return torch.version.cuda is not None


def compile_module(build_dir, verbose=False):
    import sysconfig

    import torch

    base = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    obj = os.path.join(build_dir, TORCH_SOURCE.replace(".cpp", ".o"))
    _run(["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-I", INCLUDE, "-isystem", base, "-isystem", os.path.join(base, "torch", "csrc", "api", "include"),
          "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda, "-c", os.path.join(CSRC, TORCH_SOURCE),
          "-o", obj], verbose, f"g++ on {TORCH_SOURCE}")
    return obj


def link_module(obj, verbose=False):
    import torch

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = TORCH_LIB_PATH + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, "-L" + HERE, "-l:" + os.path.basename(LIB_PATH), "-L" + lib, "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10",
          "-lc10_cuda", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib], verbose, "link of _csa_torch.so")
    os.replace(tmp, TORCH_LIB_PATH)


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
