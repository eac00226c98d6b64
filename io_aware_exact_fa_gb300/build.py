"""Build libfa_gb300.so in-tree with nvcc for sm_103a (no cmake, no torch), and, where torch, its headers, Python's and a C++
compiler are there, the binding's compiled part _binding.so. Without that part the binding makes the same calls in Python, with
about twice the time on the host.

    python -m io_aware_exact_fa_gb300.build [--verbose] [--ptxas-info] [--debug]

Compiles the translation units under csrc/ in parallel into _build/ and
links them (static CUDA runtime) into io_aware_exact_fa_gb300/libfa_gb300.so.
With --debug (debug=True) the same sources are compiled with FA_DEBUG=1 into
_build_debug/ and libfa_gb300_debug.so: the device-checking build.
Rebuilds only when a source or header is newer than the library.
"""

from __future__ import annotations

import argparse
import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libfa_gb300.so")
LIB_DEBUG = os.path.join(PKG, "libfa_gb300_debug.so")
BINDING = os.path.join(PKG, "_binding.so")   # argument checks of the paged calls
BINDING_STAMP = os.path.join(BUILD, "binding.torch")   # the torch that it was built against
SOURCES = ["fa_api.cu", "prefill_sm103.cu", "decode_sm103.cu", "backward_sm103.cu", "decode_grouped_sm103.cu",
           "materialized_sm103.cu", "append_paged_sm103.cu", "decode_paged_sm103.cu",
           "read_paged_sm103.cu", "weigh_paged_sm103.cu", "evict_paged_sm103.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put it on PATH)")


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return files


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(f) <= t for f in _deps())


def _build_binding(force: bool) -> bool:
    """Builds _binding.so; False, with a line on stderr and no old one left, where that is not possible."""
    try:
        _compile_binding(force)
        return True
    except Exception as e:   # (the library does not need it)
        sys.stderr.write(f"_binding.so was not built ({e}): the paged calls check their arguments in Python\n")
        for old in (BINDING, BINDING_STAMP):
            if os.path.exists(old):
                os.remove(old)
        return False


def _compile_binding(force: bool) -> None:
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("no torch")
    torch = os.path.realpath(list(spec.submodule_search_locations)[0])
    with open(os.path.join(torch, "version.py")) as f:
        built_with = torch + "\n" + sys.version + "\n" + f.read()
    if not force and up_to_date(BINDING) and os.path.exists(BINDING_STAMP):
        with open(BINDING_STAMP) as f:
            if f.read() == built_with:
                return
    os.makedirs(BUILD, exist_ok=True)
    tmp = BINDING + ".tmp"
    cmd = [os.environ.get("CXX") or shutil.which("g++") or "c++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", INCLUDE, "-I",
           os.path.join(torch, "include"), "-I", sysconfig.get_paths()["include"], os.path.join(CSRC, "binding.cpp"), "-o", tmp,
           "-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if os.path.exists(os.path.join(torch, "lib", "libtorch_cuda.so")):   # (else nothing is ever allocated on a GPU)
        cmd += ["-DFA_TORCH_CUDA", "-Wl,--no-as-needed", "-ltorch_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        raise RuntimeError("the C++ compiler failed on binding.cpp")
    os.replace(tmp, BINDING)
    with open(BINDING_STAMP, "w") as f:
        f.write(built_with)


def build(verbose: bool = False, ptxas_info: bool = False, force: bool = False, debug: bool = False) -> str:
    """Compile and link the library (the checking build with debug=True); returns its path."""
    lib = LIB_DEBUG if debug else LIB
    bdir = BUILD + "_debug" if debug else BUILD
    binding = lambda: None if debug else _build_binding(force)   # noqa: E731
    if not force and not ptxas_info and up_to_date(lib):
        binding()
        return lib
    os.makedirs(bdir, exist_ok=True)
    cc = nvcc()
    flags = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
                    "--expt-relaxed-constexpr"] + (["-DFA_DEBUG=1"] if debug else [])
    if ptxas_info:
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(bdir, src.replace(".cu", ".o"))
        cmd = [cc, "-c", os.path.join(CSRC, src), "-o", obj] + flags
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, cmd, r

    objs = []
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        bound = ex.submit(binding)
        for src, obj, cmd, r in ex.map(compile_one, SOURCES):
            if verbose or ptxas_info or r.returncode != 0:
                sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed on {src}")
            objs.append(obj)
        bound.result()
    tmp = lib + ".tmp"
    # cuBLAS (the materialising baseline's GEMMs) is opened at run time with dlopen, not linked
    cmd = [cc, "-shared", "-o", tmp] + objs + ARCH + ["-cudart", "static", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError("link failed")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true")
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--debug", action="store_true", help="the device-checking build (FA_DEBUG=1)")
    a = ap.parse_args()
    print(build(a.verbose, a.ptxas_info, a.force, a.debug))
