"""Build the CUDA library in-tree: paged_kv_gqa_14_gb300/_build/libpkv.so (sm_103a only).

Each translation unit is compiled by its own nvcc process in parallel, then linked into a
shared library against the shared CUDA runtime.  Beside it a CPython extension in plain C (q8_call.c), named for the
interpreter that it is built for; where it does not compile (no C compiler, no Python headers) the library is built
all the same, and the calls that need the extension say that it is missing.  Rebuilds only what is older than a source
or header.  ``python -m paged_kv_gqa_14_gb300.build [--force] [--verbose]``.
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
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libpkv.so")
# the Python side of the 8-bit cache's calls, for this interpreter's ABI
CALL = os.path.join(BUILD, "_q8call" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

# (source, object name, extra flags): decode_tc.cu is built once per pool block size
SOURCES = [("abi.cu", "abi.o", []), ("kv_append.cu", "kv_append.o", []), ("attention.cu", "attention.o", []),
           ("noalloc.cu", "noalloc.o", []), ("copy.cu", "copy.o", []), ("kv_q8.cu", "kv_q8.o", []),
           ("decode_q8.cu", "decode_q8.o", []), ("prefill_q8.cu", "prefill_q8.o", [])] + [
    ("decode_tc.cu", f"decode_tc_bs{bs}.o", [f"-DPKV_DECODE_TC_BS={bs}"]) for bs in (8, 16, 32, 64, 128)]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
# No --use_fast_math: sincosf in the RoPE kernel stays the accurate library routine; the
# kernels call fast approximations (ex2.approx) explicitly where they want them.
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden"]


def nvcc():
    exe = shutil.which("nvcc")
    if exe:
        return exe
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def c_compiler():
    return shutil.which("gcc") or shutil.which("cc") or "cc"


def _newer_than(built, sources):
    return os.path.exists(built) and all(os.path.getmtime(f) <= os.path.getmtime(built) for f in sources)


def _lib_up_to_date():
    files = [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC)) if f.endswith((".cu", ".cuh", ".h"))]
    return _newer_than(LIB, [os.path.join(INCLUDE, "pkv.h"), *files])


def _call_up_to_date():
    return _newer_than(CALL, [os.path.join(INCLUDE, "pkv.h"), os.path.join(CSRC, "q8_call.c")])


def _start_call(verbose):
    """The extension's compiler process; None where there is no compiler."""
    cmd = [c_compiler(), "-O2", "-std=c11", "-shared", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE, "-I",
           sysconfig.get_paths()["include"], os.path.join(CSRC, "q8_call.c"), "-o", CALL + ".tmp"]
    if verbose:
        print(" ".join(cmd), flush=True)
    try:
        return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    except OSError as e:
        print(f"--- q8_call.c\n{e}", flush=True)
        return None


def _finish_call(p, verbose):
    out = p.communicate()[0] if p else ""
    if out and (verbose or p.returncode):
        print(f"--- q8_call.c\n{out}", flush=True)
    if p and p.returncode == 0:
        os.replace(CALL + ".tmp", CALL)
        return
    if os.path.exists(CALL):  # (built from older sources)
        os.remove(CALL)
    print("warning: the extension for the 8-bit cache's calls from Python is not built (it needs a C compiler and "
          "Python's headers)", flush=True)


def build(force=False, verbose=False, ptxas_info=False):
    """Compile and link; returns the library path."""
    os.makedirs(BUILD, exist_ok=True)
    call = None
    need_call = force or not _call_up_to_date()
    if need_call:
        call = _start_call(verbose)
    try:
        if force or not _lib_up_to_date():
            _build_lib(verbose, ptxas_info)
    finally:
        if need_call:
            _finish_call(call, verbose)
    return LIB


def _build_lib(verbose, ptxas_info):
    cc = nvcc()
    procs = []
    objs = []
    for src, oname, extra in SOURCES:
        obj = os.path.join(BUILD, oname)
        cmd = [cc, *ARCH, *FLAGS, *extra, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", obj]
        if ptxas_info:
            cmd += ["-Xptxas", "-v"]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((oname, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
        objs.append(obj)
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if out and (verbose or ptxas_info or p.returncode):
            print(f"--- {src}\n{out}", flush=True)
        if p.returncode:
            failed.append(src)
    if failed:
        raise RuntimeError(f"compilation failed for {failed}")
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
