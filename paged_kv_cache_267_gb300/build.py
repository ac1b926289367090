"""Builds libpa.so in-tree: CUDA kernels for sm_103a with nvcc, host C++ with
g++, one shared library with the C ABI declared in include/pa.h; and next to it
_pa_torch.so, the binding of the hot calls for torch tensors (pa_torch.cpp).

Translation units compile in parallel; the library is rebuilt only when a
source, header or this script is newer than it.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libpa.so")
BINDING_PATH = os.path.join(PKG, "_pa_torch.so")
BINDING_STAMP = os.path.join(BUILD_DIR, "pa_torch.stamp")  # the torch it was built for

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CU_SOURCES = ["decode_bf16.cu", "decode_f16.cu", "decode_fp8.cu", "decode_mq_bf16.cu",
              "decode_mq_f16.cu", "decode_mq_fp8.cu", "chunk_tc.cu", "merge_reshape.cu",
              "decode_noalloc.cu", "selftest.cu", "pool_ops.cu", "norm_cache.cu",
              "shared_plan.cu", "prefix_tc.cu", "shared_merge.cu", "decode_sh_bf16.cu", "decode_sh_f16.cu",
              "decode_sh_fp8.cu", "packed_plan.cu", "packed_tc.cu", "packed_tc_small.cu",
              "packed_tc_whole.cu", "packed_merge.cu", "cache_moves.cu"]
CPP_SOURCES = ["pa_api.cpp", "pa_step.cpp", "pa_packed.cpp", "pa_alloc.cpp"]


def cuda_home() -> str:
    for c in (os.environ.get("CUDA_HOME"), os.environ.get("CUDA_PATH"), "/usr/local/cuda"):
        if c and os.path.exists(os.path.join(c, "bin", "nvcc")):
            return c
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(nvcc))
    raise RuntimeError("nvcc not found: set CUDA_HOME")


def _deps() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    return files + [os.path.join(INCLUDE, "pa.h"), os.path.abspath(__file__)]


def _binding_stamp() -> str:
    import torch
    return f"{torch.__version__} {sysconfig.get_config_var('SOABI')}"


def binding_fits() -> bool:
    """Whether _pa_torch.so was built for this torch and Python."""
    try:
        with open(BINDING_STAMP, encoding="utf-8") as f:
            return os.path.exists(BINDING_PATH) and f.read() == _binding_stamp()
    except OSError:
        return False


def is_stale() -> bool:
    if not os.path.exists(LIB_PATH) or not binding_fits():
        return True
    t = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(p) > t for p in _deps())


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and not is_stale():
        return LIB_PATH
    home = cuda_home()
    nvcc = os.path.join(home, "bin", "nvcc")
    os.makedirs(BUILD_DIR, exist_ok=True)
    jobs, objs = [], []
    for src in CU_SOURCES:
        obj = os.path.join(BUILD_DIR, src + ".o")
        cmd = [nvcc, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
               "-I", INCLUDE, "-c", os.path.join(CSRC, src), "-o", obj]
        jobs.append((src, cmd))
        objs.append(obj)
    for src in CPP_SOURCES:
        obj = os.path.join(BUILD_DIR, src + ".o")
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-I", INCLUDE,
               "-I", os.path.join(home, "include"), "-c", os.path.join(CSRC, src), "-o", obj]
        jobs.append((src, cmd))
        objs.append(obj)
    import torch
    tdir = os.path.dirname(torch.__file__)
    binding_obj = os.path.join(BUILD_DIR, "pa_torch.cpp.o")
    jobs.append(("pa_torch.cpp", [
        "g++", "-O2", "-std=c++17", "-fPIC",
        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
        "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(tdir, "include"),
        "-isystem", os.path.join(tdir, "include", "torch", "csrc", "api", "include"),
        "-isystem", os.path.join(home, "include"), "-c", os.path.join(CSRC, "pa_torch.cpp"),
        "-o", binding_obj]))
    procs = [(src, cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT))
             for src, cmd in jobs]
    failed = []
    for src, cmd, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append((src, out.decode(errors="replace")))
        elif verbose and out:
            sys.stdout.write(out.decode(errors="replace"))
    if failed:
        msg = "\n".join(f"--- {s}\n{o}" for s, o in failed)
        raise RuntimeError(f"libpa build failed:\n{msg}")
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    link = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lpthread", "-ldl"]
    r = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError("libpa link failed:\n" + r.stdout.decode(errors="replace"))
    os.replace(tmp, LIB_PATH)
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    tlib = os.path.join(tdir, "lib")
    link = ["g++", "-shared", "-o", tmp, binding_obj, "-L", PKG, "-l:libpa.so", "-L", tlib,
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN",
            f"-Wl,-rpath,{tlib}"]
    r = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError("binding link failed:\n" + r.stdout.decode(errors="replace"))
    os.replace(tmp, BINDING_PATH)
    with open(BINDING_STAMP, "w", encoding="utf-8") as f:
        f.write(_binding_stamp())
    return LIB_PATH


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose=True))
