"""Compile the CUDA library (csrc/*.cu) into _lib/librs.so for sm_103a.

One translation unit per key type plus the C-ABI unit, compiled in parallel
with nvcc, then linked into a shared library with the CUDA runtime linked
statically.  Beside it, csrc/rs_torch.cpp becomes a CPython extension for the
installed torch (the expert operators' calls without the interpreter's cost;
skipped where torch has no CUDA, and with a warning where it does not build:
the calls then go through Python).  Nothing here runs at import time of the
package except the check that the library exists.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIBDIR = os.path.join(HERE, "_lib")
LIB = os.path.join(LIBDIR, "librs.so")
INCLUDE = os.path.join(ROOT, "include")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")
    return path


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def torch_dir() -> str | None:
    """The installed torch's folder if it has CUDA (found without importing it)."""
    spec = importlib.util.find_spec("torch")
    root = spec and spec.submodule_search_locations and list(spec.submodule_search_locations)[0]
    return root if root and os.path.exists(os.path.join(root, "lib", "libc10_cuda.so")) else None


def torch_ext() -> str | None:
    """Path of the extension for this Python and the installed torch (built or not)."""
    if not torch_dir():
        return None
    return os.path.join(LIBDIR, f"rs_torch_{importlib.metadata.version('torch')}.{sysconfig.get_config_var('SOABI')}.so")


def build_torch_ext(force: bool = False) -> str | None:
    """Build the extension if a source is newer than it; its path, or None
    where there is none.  The library does not need it, so what keeps it from
    being built is a warning."""
    out, src = torch_ext(), os.path.join(CSRC, "rs_torch.cpp")
    if out is None:
        return None
    deps = [src, *glob.glob(os.path.join(INCLUDE, "*.h"))]
    if not force and os.path.exists(out) and os.path.getmtime(out) >= max(map(os.path.getmtime, deps)):
        return out
    os.makedirs(LIBDIR, exist_ok=True)
    root, tmp = torch_dir(), out + f".{os.getpid()}.tmp"
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", os.path.join(root, "include"), "-I",
           os.path.join(root, "include", "torch", "csrc", "api", "include"), "-I", cuda, "-I",
           sysconfig.get_paths()["include"], "-I", INCLUDE, src, "-L", os.path.join(root, "lib"), "-ltorch_python",
           "-ltorch_cpu", "-lc10", "-lc10_cuda", "-o", tmp]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        why = "" if r.returncode == 0 else f"{r.stdout}\n{r.stderr}"
    except OSError as e:
        why = str(e)
    if why:
        if os.path.exists(out):  # of older sources: its structures may not be the library's
            os.remove(out)
        warnings.warn(f"the expert operators' extension was not built, their calls go through Python: g++ failed on "
                      f"{src}:\n{why}", RuntimeWarning, stacklevel=2)
        return None
    os.replace(tmp, out)
    return out


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
    deps += glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, extra_flags=(), verbose: bool = False, libdir: str | None = None) -> str:
    """Build librs.so if any source is newer than it; returns its path.

    extra_flags / libdir build a variant (e.g. -D switches) into another folder.
    """
    out_dir = libdir or LIBDIR
    out_lib = os.path.join(out_dir, "librs.so")
    if not force and libdir is None and not _stale():
        build_torch_ext()
        return LIB
    os.makedirs(out_dir, exist_ok=True)
    objdir = os.path.join(out_dir, "obj")
    os.makedirs(objdir, exist_ok=True)
    common = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-I", INCLUDE, "-I", CSRC, *extra_flags]

    def compile_one(src):
        obj = os.path.join(objdir, os.path.basename(src)[:-3] + ".o")
        cmd = common + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(16, os.cpu_count() or 1)) as ex:
        ext = ex.submit(build_torch_ext, force) if libdir is None else None
        objs = list(ex.map(compile_one, sources()))
        if ext:
            ext.result()
    tmp = out_lib + f".{os.getpid()}.tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out_lib)
    return out_lib


if __name__ == "__main__":
    # python -m lsd_radix_sort_key_gb300._build [--libdir DIR --flags "-DNAME=VALUE ..."]
    # builds the library, or a variant of it (compile-time switches, e.g. the
    # shapes in rs_config.h) into DIR, and prints the library's path.
    import argparse
    import shlex
    ap = argparse.ArgumentParser()
    ap.add_argument("--libdir", default=None)
    ap.add_argument("--flags", default="")
    a = ap.parse_args()
    print(build(force=True, verbose=True, extra_flags=shlex.split(a.flags), libdir=a.libdir))
