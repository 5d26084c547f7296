"""Builds libreplayssm.so in-tree with nvcc for sm_103a, and _blockcall.so, the
C++ side of block.py's calls, with g++ against the installed torch.

Each translation unit compiles in its own nvcc process (in parallel), then
nvcc links them into one shared library (CUDA runtime linked statically).
"""
import concurrent.futures
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libreplayssm.so")
SOURCES = ["rsm_api.cu", "rsm_inst_f32.cu", "rsm_inst_bf16.cu", "rsm_inst_f16.cu", "rsm_inst_q8.cu", "rsm_inst_q8sr.cu",
           "rsm_inst_tc.cu", "rsm_inst_q8tc.cu", "gdn_inst.cu", "block_api.cu", "ssm_inst.cu", "ssm_tc_inst.cu", "ssm_token_bf16.cu", "ssm_token_f32.cu",
           "norm_inst.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
              "-I", os.path.join(ROOT, "include"), "--expt-relaxed-constexpr"]


CALL_SOURCE = os.path.join(CSRC, "blockcall.cpp")
CALL_LIB = os.path.join(PKG, "_blockcall.so")


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libreplayssm.so")


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if os.path.join(CSRC, f) != CALL_SOURCE]
    files += [os.path.join(ROOT, "include", f) for f in ("replayssm.h", "replayssm_block.h")]
    files += [os.path.abspath(__file__)]
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    return os.path.getmtime(LIB) >= max(os.path.getmtime(f) for f in _deps())


def build_calls(force: bool = False, verbose: bool = False) -> str:
    """Compiles _blockcall.so: a Python extension on torch's C++ tensors."""
    import sysconfig

    import torch
    deps = [CALL_SOURCE, os.path.abspath(__file__), torch.__file__]
    deps += [os.path.join(ROOT, "include", f) for f in ("replayssm.h", "replayssm_block.h")]
    if not force and os.path.exists(CALL_LIB) and os.path.getmtime(CALL_LIB) >= max(os.path.getmtime(f) for f in deps):
        return CALL_LIB
    at = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = CALL_LIB + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
           "-I", os.path.join(at, "include"), "-I", os.path.join(at, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(cuda, "include"), "-I", sysconfig.get_paths()["include"], CALL_SOURCE, "-o", tmp,
           "-L" + os.path.join(at, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on blockcall.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALL_LIB)
    return CALL_LIB


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and not extra_flags and up_to_date():
        build_calls(False, verbose)
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = ex.submit(build_calls, force, verbose)
        objs = list(ex.map(compile_one, SOURCES))
        calls.result()
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [cc, *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    extra = [a for a in sys.argv[1:] if a.startswith("-") and a not in ("--force", "-v")]
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, extra_flags=extra))
