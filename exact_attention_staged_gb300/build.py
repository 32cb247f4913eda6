"""Build libfa.so in-tree with nvcc for sm_103a (one -gencode, translation units in parallel), and
the Python extension beside it with the host compiler.

Usage: ``python -m exact_attention_staged_gb300.build`` or ``build()`` from Python.
Objects go to ``exact_attention_staged_gb300/_build/``; the library to
``exact_attention_staged_gb300/libfa.so``, the extension to ``_binding`` with the interpreter's own
suffix, so that no other Python version loads it.  All are git-ignored.
"""
from __future__ import annotations

import concurrent.futures
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
LIB = os.path.join(PKG, "libfa.so")
# Python extension: the short calls' per-call path
BINDING = os.path.join(PKG, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
SOURCES = ["fa_api.cu", "fa_fwd.cu", "fa_fwd_fp8.cu", "fa_bwd.cu", "fa_decode.cu", "fa_rope.cu",
           "fa_paged.cu", "fa_paged_attn.cu", "fa_pages.cu", "fa_beam.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfa.so")


def _flags():
    return ["-std=c++17", "-O3", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC",
            "-I", INCLUDE, "-I", CSRC]


def _stale(target: str, sources) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    deps = [os.path.join(CSRC, f) for f in sources] + [os.path.join(INCLUDE, "fa.h"), __file__]
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Build what is out of date; returns the library's path.

    The library does not depend on the extension: where that does not compile (no Python headers, no
    host compiler), its error is printed and the calls that need it raise.
    """
    need_lib = force or _stale(LIB, [f for f in os.listdir(CSRC) if f != "binding.c"])
    need_binding = force or _stale(BINDING, ["binding.c"])
    if not need_lib and not need_binding:
        return LIB
    nvcc = _nvcc() if need_lib else ""
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc, *_flags(), "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{res.stdout}\n{res.stderr}")
        if verbose and (res.stdout or res.stderr):
            print(res.stdout + res.stderr, file=sys.stderr)
        return obj

    def compile_binding() -> None:
        tmp = BINDING + f".tmp{os.getpid()}"
        cmd = [shutil.which("gcc") or "cc", "-O2", "-std=c11", "-Wall", "-fPIC", "-shared",
               "-I", sysconfig.get_path("include"), "-I", INCLUDE, os.path.join(CSRC, "binding.c"),
               "-o", tmp, "-lm"]
        try:
            res = subprocess.run(cmd, capture_output=True, text=True)
            error = f"{res.stdout}\n{res.stderr}" if res.returncode != 0 else None
        except OSError as e:
            error = str(e)
        if error is None:
            os.replace(tmp, BINDING)
            return
        if os.path.exists(BINDING):  # of older sources
            os.remove(BINDING)
        print(f"compiling binding.c failed, the calls that need it will raise:\n{error}",
              file=sys.stderr)

    def link(objs) -> None:
        tmp = LIB + f".tmp{os.getpid()}"
        res = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True,
                             text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, LIB)

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(compile_binding) if need_binding else None
        if need_lib:
            link(list(ex.map(compile_one, SOURCES)))
        if binding is not None:
            binding.result()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
