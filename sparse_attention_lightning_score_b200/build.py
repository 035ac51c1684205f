"""Build ``libli.so`` in-tree with nvcc for sm_100a (no GPU needed to compile).

    python -m sparse_attention_lightning_score_b200.build [--force] [--verbose] [--abi-only]

Every ``csrc/*.cu`` is compiled to an object with
``-gencode arch=compute_100a,code=sm_100a -lineinfo -O3`` and the objects are
linked into ``libli.so`` (CUDA runtime linked statically; the driver is reached
through the runtime's entry-point query, so no libcuda link is needed).
That needs nvcc alone.  ``csrc/bind.cpp`` is then compiled against the installed
torch (its headers, ``Python.h``, g++) into ``_bind.so``, the binding of the
paged-cache calls, which calls ``libli.so`` beside it; again whenever torch or
Python is another one.  ``--abi-only`` (``build(bind=False)``) leaves it out; where
there is no torch, this file is run by its path, as the package imports torch.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libli.so")
BIND_SRC = os.path.join(CSRC, "bind.cpp")
BIND = os.path.join(PKG, "_bind.so")
BIND_STAMP = os.path.join(BUILD_DIR, "bind.txt")  # what _bind.so was built against

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
                     "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found: the li CUDA library cannot be built")
    return p


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _run(cmd, verbose=False):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout, r.stderr, file=sys.stderr)


def build(force: bool = False, verbose: bool = False, extra_flags=None, bind: bool = True) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    hdrs = _headers()
    objs = []
    jobs = []
    for src in _sources():
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + hdrs):
            cmd = [nvcc()] + NVCC_FLAGS + (extra_flags or []) + ["-c", src, "-o", obj]
            jobs.append(cmd)

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        # (the binding's compilation takes as long as the kernels': both at once)
        binding = ex.submit(_bind_object, force, verbose) if bind else None
        list(ex.map(lambda cmd: _run(cmd, verbose), jobs))
        if force or jobs or _stale(LIB, objs):
            _run([nvcc()] + ARCH + ["-shared", "-o", LIB] + objs, verbose)
        if binding is not None:
            _bind_library(*binding.result(), verbose)  # raises what its compilation raised; libli.so is there by now
    return LIB


def _bind_object(force, verbose):
    """bind.o, compiled if need be: (its path, what it was built against, whether it is new)."""
    try:
        import torch
        against = "\n".join([sys.version, torch.__version__, str(torch.version.git_version), torch.__file__,
                             str(torch._C._GLIBCXX_USE_CXX11_ABI)])
    except ImportError as e:
        raise RuntimeError("libli.so needs nvcc alone (--abi-only); its PyTorch binding _bind.so needs torch") from e
    obj = os.path.join(BUILD_DIR, "bind.o")
    try:
        with open(BIND_STAMP) as f:
            same = f.read() == against
    except OSError:
        same = False
    new = force or not same or _stale(obj, [BIND_SRC] + _headers())
    if new:
        if os.path.exists(BIND_STAMP):
            os.remove(BIND_STAMP)  # (until the library of this object is there)
        _run(_bind_compile(obj), verbose)
    return obj, against, new


def _bind_library(obj, against, new, verbose):
    if new or _stale(BIND, [obj]):
        _run(_bind_link(obj), verbose)
        with open(BIND_STAMP, "w") as f:
            f.write(against)


def _bind_compile(obj):
    """g++ command for bind.cpp (torch's headers, its C++ ABI)."""
    import sysconfig
    import torch
    from torch.utils import cpp_extension
    inc = [f"-I{d}" for d in cpp_extension.include_paths(device_type="cuda") + [sysconfig.get_path("include"), INCLUDE]]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-Wno-unknown-pragmas",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"] + inc + ["-c", BIND_SRC, "-o", obj]


def _bind_link(obj):
    from torch.utils import cpp_extension
    libs = cpp_extension.library_paths(device_type="cuda")
    return (["g++", "-shared", "-o", BIND, obj, f"-L{PKG}", "-lli"] + [f"-L{d}" for d in libs] +
            ["-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"] +
            [f"-Wl,-rpath,{d}" for d in libs[:1]])


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print register/spill/smem usage per kernel")
    ap.add_argument("--abi-only", action="store_true", help="libli.so alone, without the PyTorch binding")
    args = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if args.ptxas_info else None
    print(build(force=args.force or args.ptxas_info, verbose=args.verbose or args.ptxas_info, extra_flags=extra,
                bind=not args.abi_only))


if __name__ == "__main__":
    main()
