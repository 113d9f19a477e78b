"""Compile libdspark.so in-tree with nvcc for sm_103a (one -gencode, parallel compiles), and _native.so, the
CPython module of the paged-cache calls (g++, against torch's headers)."""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libdspark.so")
NATIVE = os.path.join(HERE, "_native.so")
SOURCES = ["api.cu", "sample.cu", "sample_tc.cu", "verify.cu", "tv.cu", "schedule.cu", "logits.cu", "cache.cu",
           "paged_attn.cu", "paged_attn_tc.cu"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc" if os.path.exists("/usr/local/cuda/bin/nvcc") else "nvcc")
FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
         "-I", INCLUDE, "-I", CSRC]


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(NATIVE):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(NATIVE))
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "dspark.h"), os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps)


def _native_command(obj: str) -> list[str]:
    """g++ command that compiles native.cpp to `obj`."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    inc = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"], INCLUDE,
           os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include") if os.path.isabs(NVCC) else "/usr/local/cuda/include"]
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return ["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={abi}", *[f for i in inc for f in ("-I", i)], "-c",
            os.path.join(CSRC, "native.cpp"), "-o", obj]


def _link_native(obj: str) -> None:
    import torch

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = NATIVE + f".tmp{os.getpid()}"
    subprocess.check_call(["g++", "-shared", "-o", tmp, obj, LIB, "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
                           "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"])
    os.replace(tmp, NATIVE)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        cmd = [NVCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        return obj, r.stderr

    def compile_native():
        obj = os.path.join(objdir, "native.o")
        r = subprocess.run(_native_command(obj), capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed for native.cpp:\n{r.stderr}")
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        native = ex.submit(compile_native)
        results = list(ex.map(compile_one, SOURCES))
        native_obj = native.result()
    if verbose:
        for _, err in results:
            print(err)
    tmp = LIB + f".tmp{os.getpid()}"
    # (with a name of its own, so that _native.so asks for it by that and finds it beside itself, wherever the tree is)
    subprocess.check_call([NVCC, "-shared", "-gencode", "arch=compute_103a,code=sm_103a", "-cudart", "shared",
                           "-Xlinker", "-soname=" + os.path.basename(LIB), "-o", tmp, *[o for o, _ in results]])
    os.replace(tmp, LIB)
    _link_native(native_obj)
    return LIB


if __name__ == "__main__":
    import sys

    print(build(force=True, verbose="-v" in sys.argv))
