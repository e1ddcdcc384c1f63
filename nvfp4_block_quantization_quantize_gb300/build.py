"""Builds the sm_103a library ``libnvfp4_gb300.so`` in-tree with nvcc.

Each translation unit compiles in parallel with ``-gencode
arch=compute_103a,code=sm_103a`` (GB300 only), then one shared library is
linked with the static CUDA runtime.  Beside them g++ compiles
``_nvfp4_call``, the binding's short path for the serving operators (CPython
and torch headers; it holds no arithmetic), which is made again for another torch
or interpreter.  The fp32 steps the method pins must
round exactly as written, so the build keeps IEEE division / square root,
does not flush subnormals and does not contract multiply-adds.
"""
from __future__ import annotations

import concurrent.futures as cf
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
LIB_PATH = os.path.join(PKG, "libnvfp4_gb300.so")
CALL_PATH = os.path.join(PKG, "_nvfp4_call" + sysconfig.get_config_var("EXT_SUFFIX"))
CALL_ABI_PATH = os.path.join(BUILD_DIR, "_nvfp4_call.abi")      # what CALL_PATH was built for
SOURCES = ["nvfp4_rows.cu", "nvfp4_tiles.cu", "nvfp4_aux.cu", "nvfp4_mm.cu", "nvfp4_norm.cu", "nvfp4_mv.cu",
           "nvfp4_grouped.cu", "nvfp4_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-ftz=false",
         "-prec-div=true", "-prec-sqrt=true", "-fmad=false", "-I", INCLUDE]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libnvfp4_gb300.so")


def call_abi() -> str:
    """The torch and the interpreter that the short path is compiled against (it uses their C++ and C layouts)."""
    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def _call_command(out: str) -> list[str]:
    import torch
    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [INCLUDE, os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    libs = ["torch_python", "torch_cuda", "torch_cpu", "c10_cuda", "c10"]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++20", "-fPIC", "-shared", f'-DNVFP4_CALL_ABI="{call_abi()}"',
            *[f"-I{i}" for i in inc], os.path.join(CSRC, "nvfp4_call.cpp"), "-o", out, "-L" + os.path.join(t, "lib"), *["-l" + n for n in libs],
            "-Wl,-rpath," + os.path.join(t, "lib")]


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "nvfp4.h"))
    files.append(os.path.abspath(__file__))
    return files


def source_digest() -> str:
    """sha256 over the kernel sources and the ABI header (identifies a build)."""
    import hashlib
    h = hashlib.sha256()
    for f in sorted(os.listdir(CSRC)):
        h.update(f.encode())
        h.update(open(os.path.join(CSRC, f), "rb").read())
    h.update(open(os.path.join(INCLUDE, "nvfp4.h"), "rb").read())
    return h.hexdigest()[:16]


def is_stale() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(CALL_PATH):
        return True
    if not os.path.exists(CALL_ABI_PATH) or open(CALL_ABI_PATH).read() != call_abi():
        return True
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(CALL_PATH))
    return any(os.path.getmtime(f) > t for f in _deps())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and not is_stale():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        return obj, r.stderr

    def compile_call():
        tmp = os.path.join(BUILD_DIR, f"_nvfp4_call.tmp{os.getpid()}")
        r = subprocess.run(_call_command(tmp), capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on nvfp4_call.cpp:\n{r.stderr}")
        return tmp

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        call = ex.submit(compile_call)
        results = list(ex.map(compile_one, SOURCES))
    if verbose or ptxas_info:
        for obj, log in results:
            sys.stderr.write(log)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    os.replace(call.result(), CALL_PATH)        # last: the library is there without it
    with open(CALL_ABI_PATH, "w") as f:
        f.write(call_abi())
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
