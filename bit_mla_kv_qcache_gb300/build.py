"""Compile the CUDA library (csrc/*.cu -> libmla_qcache.so) for sm_103a with nvcc, in tree."""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmla_qcache.so")
FAST = os.path.join(PKG, "_fastcall" + sysconfig.get_config_var("EXT_SUFFIX"))  # native argument marshalling
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
SOURCES = {  # file -> extra flags
    "abi.cu": [],
    "writer.cu": ["-fmad=false"],  # exact rounding decisions: keep every product unfused
    "decode.cu": [],
    "decode_tc.cu": [],
    "proj.cu": [],
    "diag.cu": [],
    "abi_kv4.cu": [],
    "kv4_append.cu": ["-fmad=false"],  # as the writer
    "kv4_attn.cu": [],
    "kv4_prompt.cu": [],
    "latent_append.cu": [],
}


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")
    return cand


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(FAST):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(FAST))
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(ROOT, "include", "mla_qcache.h"),
                                                                  __file__]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    common = ["-std=c++17", "-O3", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"),
              "-diag-suppress", "177"]

    def compile_one(item):
        src, extra = item
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc, *common, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd))
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj

    def compile_fast():
        import torch
        from torch.utils import cpp_extension
        obj = os.path.join(BUILD, "fastcall.o")
        cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
        inc = [sysconfig.get_paths()["include"], os.path.join(ROOT, "include"), os.path.join(cuda, "include"),
               *cpp_extension.include_paths()]
        cmd = ["g++", "-std=c++17", "-O2", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
               *(x for d in inc for x in ("-isystem", d)), "-c", os.path.join(CSRC, "fastcall.cpp"), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed for fastcall.cpp:\n{r.stdout}\n{r.stderr}")
        return obj, os.path.join(os.path.dirname(torch.__file__), "lib")

    with concurrent.futures.ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        fast = ex.submit(compile_fast)
        objs = list(ex.map(compile_one, SOURCES.items()))
        fast_obj, torch_lib = fast.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc, "-shared", *ARCH, "-cudart", "shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    tmp = FAST + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, fast_obj, "-L", PKG, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN", "-L", torch_lib,
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, FAST)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
