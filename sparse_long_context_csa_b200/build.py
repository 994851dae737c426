"""Build libdsv4.so in-tree with nvcc for sm_100a (B200).

Usage: python -m sparse_long_context_csa_b200.build [--debug]
Each .cu file in csrc/ is compiled to an object in _build/ (in parallel), then linked
into sparse_long_context_csa_b200/libdsv4.so.  Objects are rebuilt when a source or a
header is newer.  csrc/binding.cpp becomes the extension module _binding.so beside it; where that
fails, a warning says so and the library is used without it.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libdsv4.so")
BINDING = os.path.join(PKG, "_binding.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def _flags(debug: bool) -> list[str]:
    f = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include"),
         "-I", CSRC, "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"] + ARCH
    if debug:
        f += ["-DDSV4_DEBUG=1"]
    return f


def _newest_header() -> float:
    hs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))
    return max((os.path.getmtime(h) for h in hs), default=0.0)


def _build_binding(hdr: float) -> None:
    """csrc/binding.cpp, which is not needed: without it abi.py makes every call through ctypes."""
    src = os.path.join(CSRC, "binding.cpp")
    if os.path.exists(BINDING) and os.path.getmtime(BINDING) > max(os.path.getmtime(src), hdr):
        return
    if os.path.exists(BINDING):  # of older sources
        os.remove(BINDING)
    torch = importlib.util.find_spec("torch")
    if torch is None:
        why = "torch is not installed"
    else:
        cmd = [os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden",
               "-I", os.path.join(ROOT, "include"), "-I", sysconfig.get_paths()["include"],
               "-I", os.path.join(torch.submodule_search_locations[0], "include"), src, "-o", BINDING]
        try:
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode == 0:
                return
            why = f"{' '.join(cmd)}\n{r.stdout}\n{r.stderr}"
        except OSError as e:
            why = str(e)
    warnings.warn(f"{os.path.basename(BINDING)} was not built, calls go through ctypes: {why}", stacklevel=3)


def build(debug: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr = _newest_header()
    flags = _flags(debug)

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        if os.path.exists(obj) and os.path.getmtime(obj) > max(os.path.getmtime(src), hdr):
            return obj, None
        cmd = [NVCC, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            return obj, f"{' '.join(cmd)}\n{r.stdout}\n{r.stderr}"
        if verbose and r.stderr.strip():
            print(r.stderr, file=sys.stderr)
        return obj, None

    with ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        results = list(ex.map(compile_one, srcs))
    errs = [e for _, e in results if e]
    if errs:
        raise RuntimeError("nvcc failed:\n" + "\n".join(errs))
    objs = [o for o, _ in results]
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        cmd = [NVCC, *ARCH, "-shared", "-o", LIB, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    _build_binding(hdr)
    return LIB


if __name__ == "__main__":
    print(build(debug="--debug" in sys.argv, verbose="-v" in sys.argv))
