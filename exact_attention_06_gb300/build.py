"""Build ``libfattn.so`` in-tree with nvcc for sm_103a.

The translation units compile in parallel into ``_build/`` and link into
``exact_attention_06_gb300/libfattn.so``; beside them the host compiler builds the
binding's module ``_calls.so`` against torch's headers, for this torch and Python only.
The library needs neither, and is linked whether or not the module compiles.
The CUDA runtime is linked statically; the driver is reached through
cudaGetDriverEntryPointByVersion, so no libcuda link is needed at build time.
"""

from __future__ import annotations

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
LIB = os.path.join(PKG, "libfattn.so")
CALLS = os.path.join(PKG, "_calls.so")
CALLS_SRC = os.path.join(CSRC, "py_calls.cpp")
CALLS_STAMP = os.path.join(BUILD, "_calls.stamp")  # what the module was built for and with
SOURCES = ["fa_fwd.cu", "fa_bwd.cu", "fa_cross_bwd.cu", "fa_cross_bwd_short.cu", "fa_cross_rows.cu", "fa_cross_short.cu",
           "fa_decode.cu", "fa_quant.cu", "fa_rope.cu", "fa_window_fwd.cu", "fa_window_bwd.cu", "fa_norm_rope.cu",
           "fa_pages.cu", "fattn_host.cu"]
GENCODE = "arch=compute_103a,code=sm_103a"


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libfattn")


def _flags():
    return ["-gencode", GENCODE, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
            "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != os.path.basename(CALLS_SRC)]
    files.append(os.path.join(INCLUDE, "fattn.h"))
    files.append(os.path.abspath(__file__))
    return files


def _newer(out: str, files) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(f) <= os.path.getmtime(out) for f in files)


def calls_abi() -> str:
    """The torch and Python whose binary interfaces the module follows; compiled into it as ``BUILT_FOR``."""
    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('EXT_SUFFIX')}"


def _cxx() -> str:
    return os.environ.get("CXX", "g++")


def _calls_key() -> str:
    import torch
    return "\n".join((calls_abi(), os.path.dirname(torch.__file__), _cxx()))


def _lib_up_to_date() -> bool:
    return _newer(LIB, _deps())


def _calls_up_to_date() -> bool:
    if not _newer(CALLS, [CALLS_SRC, os.path.join(INCLUDE, "fattn.h"), os.path.abspath(__file__)]):
        return False
    try:
        with open(CALLS_STAMP) as f:
            return f.read() == _calls_key()
    except (OSError, ImportError):
        return False


def up_to_date() -> bool:
    return _lib_up_to_date() and _calls_up_to_date()


def _calls_command(out: str):
    import torch
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    top = os.path.dirname(torch.__file__)
    inc, libs = os.path.join(top, "include"), os.path.join(top, "lib")
    return [_cxx(), "-std=c++17", "-O2", "-fPIC", "-shared", "-Wall", f'-DFATTN_BUILT_FOR="{calls_abi()}"',
            CALLS_SRC, "-o", out, "-I", INCLUDE, "-I", sysconfig.get_paths()["include"],
            "-I", cuda, "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
            f"-L{libs}", f"-Wl,-rpath,{libs}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _build_calls():
    """Compile the module; what went wrong, or None."""
    tmp = CALLS + ".tmp"
    try:
        key = _calls_key()
        r = subprocess.run(_calls_command(tmp), capture_output=True, text=True)
    except (OSError, ImportError) as e:  # no torch, no compiler
        return str(e)
    if r.returncode != 0:
        return f"{r.stdout}{r.stderr}"
    os.replace(tmp, CALLS)
    with open(CALLS_STAMP, "w") as f:
        f.write(key)
    return None


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile what is out of date, link libfattn.so; returns its path.  Raises on failure."""
    with_lib, with_calls = force or not _lib_up_to_date(), force or not _calls_up_to_date()
    if not with_lib and not with_calls:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = ex.submit(_build_calls) if with_calls else None
        if with_lib:
            _build_lib(ex, verbose, ptxas_info)
        wrong = calls.result() if calls else None
    if wrong:
        raise RuntimeError(f"{LIB} is built, the binding's module is not: py_calls.cpp:\n{wrong}")
    return LIB


def _build_lib(ex, verbose: bool, ptxas_info: bool) -> None:
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *(_flags()), *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    results = list(ex.map(compile_one, SOURCES))
    errors = []
    for src, _obj, r in results:
        if verbose or ptxas_info:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode != 0:
            errors.append(f"{src}:\n{r.stdout}{r.stderr}")
    if errors:
        raise RuntimeError("nvcc failed:\n" + "\n".join(errors))
    tmp = LIB + ".tmp"
    cmd = [cc, "-gencode", GENCODE, "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *[o for _, o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
