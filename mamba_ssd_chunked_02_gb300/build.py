"""Build the C-ABI CUDA library libmamba2_ssd.so in-tree (sm_103a only).

    python -m mamba_ssd_chunked_02_gb300.build [--force] [-j N]

Each .cu file under csrc/ is compiled by nvcc in parallel into _build/, then
linked (static CUDA runtime, no torch) into _lib/libmamba2_ssd.so.  Objects are
rebuilt when their source or any header under csrc/ or include/ is newer.

binding/layer_ext.cpp, the native Python binding of the layer operators, is
compiled by g++ beside them against the installed torch's headers and linked to
that library (_lib/layer_ext-<torch and Python>.so, a file for each pair it was
built for); without torch the library alone is built.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
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
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "libmamba2_ssd.so")
EXT_SRC = os.path.join(PKG, "binding", "layer_ext.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
                     "-DMAMBA2_SSD_BUILD", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newest_header() -> float:
    hs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(CSRC, "*.inc")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(h) for h in hs), default=0.0)


def _compile(src: str, force: bool, extra) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    if (not force and os.path.exists(obj)
            and os.path.getmtime(obj) >= max(os.path.getmtime(src), _newest_header())):
        return obj
    cmd = [nvcc()] + NVCC_FLAGS + list(extra) + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def _ext_tag() -> str:
    """What the binding's binary interface depends on: the torch and Python it is built for."""
    import torch
    return f"{torch.__version__}-{sysconfig.get_config_var('SOABI')}-cxx{int(torch._C._GLIBCXX_USE_CXX11_ABI)}"


def ext_path() -> str:
    """The Python binding for the torch and Python at hand."""
    return os.path.join(LIBDIR, f"layer_ext-{_ext_tag()}.so")


def _ext_object(force: bool) -> str | None:
    """Compile the Python binding; None without torch."""
    try:
        import torch
    except ImportError:
        return None
    obj = os.path.join(BUILD, f"layer_ext-{_ext_tag()}.o")
    newest = max(map(os.path.getmtime, glob.glob(os.path.join(os.path.dirname(EXT_SRC), "*"))))
    if not force and os.path.exists(obj) and os.path.getmtime(obj) >= max(newest, _newest_header()):
        return obj
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    dirs = [inc, os.path.join(inc, "torch", "csrc", "api", "include"), cuda,
            sysconfig.get_paths()["include"], INCLUDE]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall", "-Wextra",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += [f for d in dirs for f in ("-isystem", d)] + ["-c", EXT_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {os.path.basename(EXT_SRC)}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def _link_ext(obj: str, force: bool) -> None:
    out = ext_path()
    if not force and os.path.exists(out) and os.path.getmtime(out) >= max(os.path.getmtime(obj), os.path.getmtime(LIB)):
        return
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = out + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", LIBDIR, "-lmamba2_ssd", "-L", libs, "-ltorch_python", "-ltorch_cpu",
           "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


def build(force: bool = False, jobs: int = 0, extra=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    srcs = sources()
    jobs = jobs or min(len(srcs) + 1, os.cpu_count() or 4)
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        ext = ex.submit(_ext_object, force)
        objs = list(ex.map(lambda s: _compile(s, force, extra), srcs))
    if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc()] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    # the library is complete; the binding comes after it
    ext_obj = ext.result()
    if ext_obj:
        _link_ext(ext_obj, force)
    else:
        sys.stderr.write("torch is not installed: the Python binding of the layer operators was not built\n")
    return LIB


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-j", "--jobs", type=int, default=0)
    ap.add_argument("--ptxas-verbose", action="store_true", help="print registers / spills")
    a = ap.parse_args()
    extra = ["-Xptxas", "-v"] if a.ptxas_verbose else []
    print(build(force=a.force or a.ptxas_verbose, jobs=a.jobs, extra=extra))


if __name__ == "__main__":
    main()
