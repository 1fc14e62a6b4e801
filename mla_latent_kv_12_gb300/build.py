"""Builds libmla.so (the C-ABI library) in-tree with nvcc for sm_103a, and _native.so (the Python binding of its paged
cache) with the host compiler.

Each ``csrc/*.cu`` translation unit is compiled in parallel, then linked into
``mla_latent_kv_12_gb300/libmla.so``.  Objects go to ``_build/`` next to it.
A unit is recompiled when it, or any header under ``csrc/`` or ``include/``,
is newer than its object; the binding also when torch or Python are others
than those it was built for.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmla.so")
NATIVE = os.path.join(PKG, "_native.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-I" + os.path.join(ROOT, "include"), "-Xptxas", "-v"]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmla")
    return exe


def _headers_mtime() -> float:
    hs = glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))
    return max((os.path.getmtime(h) for h in hs), default=0.0)


def _compile(src: str, obj: str, log: str) -> tuple[str, int, str]:
    cmd = [nvcc()] + NVCC_FLAGS + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    with open(log, "w") as f:
        f.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    return src, r.returncode, r.stdout + r.stderr


def _native_tag() -> str:
    import torch
    return "\n".join((torch.__version__, os.path.dirname(torch.__file__), str(sysconfig.get_config_var("SOABI"))))


def _native_stale(obj: str, tag: str) -> bool:
    if not all(map(os.path.exists, (obj, tag, NATIVE))):
        return True
    with open(tag) as f:
        if f.read() != _native_tag():
            return True
    sources = os.path.join(CSRC, "binding.cpp"), os.path.join(ROOT, "include", "mla.h")
    return os.path.getmtime(obj) < max(map(os.path.getmtime, sources))


def _compile_native(obj: str, log: str) -> tuple[str, int, str]:
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I" + os.path.join(ROOT, "include"), "-isystem", inc, "-isystem", os.path.join(inc, "torch/csrc/api/include"),
           "-isystem", sysconfig.get_paths()["include"], "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    with open(log, "w") as f:
        f.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    return "binding.cpp", r.returncode, r.stdout + r.stderr


def _link_native(obj: str) -> None:
    import torch
    tmp = NATIVE + ".tmp"
    # torch's libraries are loaded before this one is imported; libmla.so lies beside it
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L" + PKG, "-lmla", "-Wl,-rpath,$ORIGIN",
           "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, NATIVE)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link; returns the library path.  Raises on a compile error."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr = _headers_mtime()
    jobs = []
    objs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or not os.path.exists(o) or os.path.getmtime(o) < max(os.path.getmtime(s), hdr):
            jobs.append((s, o, o + ".log"))
    native_obj = os.path.join(BUILD, "binding.o")
    native_tag = os.path.join(BUILD, "binding.tag")   # what a finished binding was built for
    native_stale = force or _native_stale(native_obj, native_tag)
    if native_stale and os.path.exists(native_tag):
        os.remove(native_tag)
    if jobs or native_stale:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs) + 1, os.cpu_count() or 4)) as ex:
            native = ex.submit(_compile_native, native_obj, native_obj + ".log") if native_stale else None
            results = list(ex.map(lambda j: _compile(*j), jobs))
            if native:
                results.append(native.result())
        bad = [(s, out) for s, rc, out in results if rc != 0]
        if bad:
            raise RuntimeError("nvcc failed:\n" + "\n".join(f"{s}:\n{out}" for s, out in bad))
        if verbose:
            for s, _, out in results:
                print(f"== {os.path.basename(s)}\n{out}")
    if force or jobs or not os.path.exists(LIB) or \
            os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        tmp = LIB + ".tmp"
        # The CUDA runtime is linked statically; the driver API (tensor maps) is
        # reached through cudaGetDriverEntryPoint, so libcuda is not a link
        # dependency and the library loads on a machine without a GPU.
        cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
        os.replace(tmp, LIB)
    if native_stale:
        _link_native(native_obj)
        with open(native_tag, "w") as f:
            f.write(_native_tag())
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
