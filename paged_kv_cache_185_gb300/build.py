"""Build libwllm.so (the sm_103a CUDA library behind include/wllm.h) and the
binding's _describe.so (calls with torch tensors) in-tree.

    python -m paged_kv_cache_185_gb300.build [--force] [--verbose]

Each translation unit is compiled by nvcc in parallel into ``_build/`` and
linked into ``paged_kv_cache_185_gb300/libwllm.so`` against the shared CUDA
runtime.  Only ``sm_103a`` code is generated.  A rebuild happens when any source
or header is newer than the library, or when _describe.so was made for another
interpreter or another torch than this process has.
"""
from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libwllm.so")
DESCRIBE = os.path.join(PKG, "_describe.so")
STAMP = os.path.join(BUILD, "describe.stamp")  # what _describe.so was made for

SOURCES = ["api.cu", "append.cu", "decode_bf16.cu", "decode_f16.cu", "decode_f32.cu", "decode_f8_f16.cu",
           "decode_f8_bf16.cu", "prefill.cu", "prefill_tc.cu", "block_manager.cpp", "api_sparse.cu", "rotate.cu",
           "rotate_f32.cu", "rotate_f16.cu", "rotate_bf16.cu", "key_bounds.cu", "select.cu", "sparse_decode.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _cuda_lib_dir(nvcc: str) -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "lib64")


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES]
    files += glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    files += glob.glob(os.path.join(CSRC, "*.inc")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    files += [os.path.join(CSRC, "describe.cpp"), os.path.abspath(__file__)]
    return files


def describe_key() -> str:
    """What _describe.so is bound to besides its source: the interpreter's ABI and the torch whose structures it reads."""
    import torch
    return f"{sysconfig.get_config_var('SOABI')} torch {torch.__version__}"


def described_for() -> str:
    """describe_key() of the build that made _describe.so ('' where nothing says)."""
    try:
        with open(STAMP) as f:
            return f.read().strip()
    except OSError:
        return ""


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(DESCRIBE)) or described_for() != describe_key():
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(DESCRIBE))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    common = [nvcc, *ARCH, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
              "-I", INCLUDE, "-I", CSRC]
    if ptxas_verbose:
        common += ["-Xptxas", "-v"]

    def compile_one(src: str):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [*common, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    # both outputs are made in _build/ and moved into place once everything is there
    lib_tmp, describe_tmp = (os.path.join(BUILD, f"{os.path.basename(f)}.{os.getpid()}.tmp") for f in (LIB, DESCRIBE))

    def describe_module():
        """The binding's CPython module: one translation unit against torch's headers."""
        import torch
        home = os.path.dirname(os.path.abspath(torch.__file__))
        libs = os.path.join(home, "lib")
        cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
               "-I", sysconfig.get_paths()["include"], "-I", os.path.join(home, "include"),
               "-I", os.path.join(home, "include", "torch", "csrc", "api", "include"),
               "-I", os.path.join(os.path.dirname(_cuda_lib_dir(nvcc)), "include"),
               os.path.join(CSRC, "describe.cpp"), "-o", describe_tmp, "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10",
               "-Wl,-rpath," + libs]
        return subprocess.run(cmd, capture_output=True, text=True)

    try:
        with ThreadPoolExecutor(len(SOURCES) + 1) as ex:
            described = ex.submit(describe_module)
            results = list(ex.map(compile_one, SOURCES))
            results.append(("describe.cpp", None, described.result()))
        failed = False
        for src, _, r in results:
            if verbose or ptxas_verbose or r.returncode != 0:
                sys.stderr.write(f"--- {src}\n{r.stdout}{r.stderr}")
            failed |= r.returncode != 0
        if failed:
            raise RuntimeError("nvcc failed")
        link = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", lib_tmp, *[o for _, o, _ in results if o is not None],
                "-Xlinker", "-rpath," + _cuda_lib_dir(nvcc), "-Xlinker", "-z,defs"]
        r = subprocess.run(link, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("link failed")
        if os.path.exists(STAMP):
            os.remove(STAMP)
        os.replace(lib_tmp, LIB)
        os.replace(describe_tmp, DESCRIBE)
        with open(STAMP, "w") as f:
            f.write(describe_key())
    finally:
        for tmp in (lib_tmp, describe_tmp):
            if os.path.exists(tmp):
                os.remove(tmp)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose, ptxas_verbose=a.ptxas_verbose))
