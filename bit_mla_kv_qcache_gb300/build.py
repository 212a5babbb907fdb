"""Compile the CUDA library (csrc/*.cu -> libmla_qcache.so) for sm_103a with nvcc, in tree."""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmla_qcache.so")
FAST_SOURCE = os.path.join(CSRC, "fastcall.cpp")
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


def _stale(target: str, sources: list) -> bool:
    if not os.path.exists(target):
        return True
    deps = [os.path.join(CSRC, f) for f in sources] + [os.path.join(ROOT, "include", "mla_qcache.h"), __file__]
    return any(os.path.getmtime(d) > os.path.getmtime(target) for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """The library and, where torch and the Python headers are at hand, the native binding (the library does not need it;
    without them a warning says so, and the entry points that go through it raise)."""
    lib_stale = force or _stale(LIB, [f for f in os.listdir(CSRC) if f != os.path.basename(FAST_SOURCE)])
    fast_stale = force or _stale(FAST, [os.path.basename(FAST_SOURCE)])
    if not lib_stale and not fast_stale:
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
        """The object and torch's libraries; None and the reason where it cannot be built."""
        try:
            import torch
            from torch.utils import cpp_extension
        except ImportError as e:
            return None, f"torch cannot be imported ({e})"
        python = sysconfig.get_paths()["include"]
        if not os.path.exists(os.path.join(python, "Python.h")):
            return None, f"no Python.h in {python}"
        obj = os.path.join(BUILD, "fastcall.o")
        cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
        inc = [python, os.path.join(ROOT, "include"), os.path.join(cuda, "include"), *cpp_extension.include_paths()]
        cmd = ["g++", "-std=c++17", "-O2", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
               *(x for d in inc for x in ("-isystem", d)), "-c", FAST_SOURCE, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed for fastcall.cpp:\n{r.stdout}\n{r.stderr}")
        return obj, os.path.join(os.path.dirname(torch.__file__), "lib")

    def link(target, cmd):
        tmp = target + ".tmp"
        r = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, target)

    with concurrent.futures.ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        fast = ex.submit(compile_fast) if fast_stale else None
        if lib_stale:
            link(LIB, [nvcc, "-shared", *ARCH, "-cudart", "shared", *ex.map(compile_one, SOURCES.items())])
        if fast:
            obj, torch_lib = fast.result()
            if obj is None:
                warnings.warn(f"the native binding is not built: {torch_lib}")
                return LIB
            link(FAST, ["g++", "-shared", obj, "-L", PKG, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN", "-L", torch_lib,
                        "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"])
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
