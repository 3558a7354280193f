"""Build ``libmoda.so`` (the C-ABI library) in-tree with nvcc for sm_100a.

Usage: ``python depth_kv_attention_b200/csrc/build.py [-v] [--force] [--ptxas-info] [--no-binding]``
(a plain script, so that it runs without importing the package, whose import
loads the library).

Each ``csrc/*.cu`` compiles to ``_build/<name>.o`` in parallel (skipped when
the object is newer than its source and every header); the objects link into
``depth_kv_attention_b200/libmoda.so``. The CUDA runtime is linked statically;
the driver entry point for tensor-map encoding is fetched at run time, so the
library needs no ``libcuda`` at link time.

``csrc/bind_torch.cpp`` (the binding of the paged-cache entry points on torch
tensors) compiles with g++ against torch's headers into
``depth_kv_attention_b200/_moda_torch.so``, which links to libmoda.so. It is
compiled again when its source, this file, torch or Python change
(``_build/moda_torch.key``). Only the paged-cache functions need it:
``--no-binding`` leaves it out, for a machine without torch's headers.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import hashlib
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

CSRC = os.path.dirname(os.path.abspath(__file__))
PKG = os.path.dirname(CSRC)
ROOT = os.path.dirname(PKG)
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmoda.so")
BIND_SRC = os.path.join(CSRC, "bind_torch.cpp")
BIND = os.path.join(PKG, "_moda_torch.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC]


def nvcc() -> str:
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found: the MoDA library needs the CUDA toolkit to build")
    return p


def _headers() -> list[str]:
    return (glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(ROOT, "include", "*.h")))


def _stale(obj: str, src: str) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(f) > t for f in [src] + _headers())


def _compile(src: str, verbose: bool, extra: list[str]) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc()] + ARCH + NVCC_FLAGS + extra + ["-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr, flush=True)
    return obj


def build(verbose: bool = False, force: bool = False, extra: list[str] | None = None,
          binding: bool = True) -> str:
    """Compile every kernel translation unit, link libmoda.so and compile the torch
    binding. Returns the library's path."""
    extra = list(extra or [])
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]
    todo = [s for s, o in zip(srcs, objs) if force or extra or _stale(o, s)]
    if todo:
        with cf.ThreadPoolExecutor(max_workers=min(8, len(todo))) as ex:
            list(ex.map(lambda s: _compile(s, verbose, extra), todo))
    if todo or not os.path.exists(LIB) or any(os.path.getmtime(o) > os.path.getmtime(LIB) for o in objs):
        cmd = [nvcc()] + ARCH + ["-shared", "-o", LIB + ".tmp"] + objs + ["-cudart", "static",
                                                                         "-Xlinker", "-soname=libmoda.so"]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(LIB + ".tmp", LIB)
    if binding:
        try:
            build_binding(verbose, force)
        except Exception as e:
            raise RuntimeError(f"{LIB} is built; the binding that the paged-cache functions need is not "
                               "(--no-binding leaves it out)") from e
    return LIB


def _binding_key() -> str:
    """What the binding is made of: its sources, this file's command, and the
    torch and Python that it is compiled against."""
    h = hashlib.sha256()
    for f in (BIND_SRC, os.path.join(ROOT, "include", "moda.h"), os.path.abspath(__file__)):
        with open(f, "rb") as fd:
            h.update(fd.read())
    torch_at = importlib.util.find_spec("torch").origin
    h.update(repr((importlib.metadata.version("torch"), torch_at, sysconfig.get_config_var("EXT_SUFFIX"))).encode())
    return h.hexdigest()


def build_binding(verbose: bool = False, force: bool = False) -> str:
    """Compile the torch binding (after libmoda.so) unless what it was made of is
    unchanged. Returns its path."""
    key_file = os.path.join(BUILD, "moda_torch.key")
    key = _binding_key()
    if not force and os.path.exists(BIND) and os.path.exists(key_file):
        with open(key_file) as f:
            if f.read() == key:
                return BIND
    import torch
    from torch.utils import cpp_extension
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    inc = cpp_extension.include_paths() + [sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            f'-DMODA_TORCH_VERSION="{torch.__version__}"']
           + [x for i in inc for x in ("-isystem", i)]
           + [BIND_SRC, "-o", BIND + ".tmp", "-L" + lib, "-ltorch", "-ltorch_cpu", "-ltorch_python", "-lc10",
              "-lc10_cuda", "-L" + PKG, "-l:libmoda.so", "-Wl,-rpath,$ORIGIN"])
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BIND_SRC}:\n{r.stdout}\n{r.stderr}")
    os.makedirs(BUILD, exist_ok=True)
    os.replace(BIND + ".tmp", BIND)
    with open(key_file, "w") as f:
        f.write(key)
    return BIND


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("-v", "--verbose", action="store_true")
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers / spills / smem")
    ap.add_argument("--no-binding", action="store_true", help="leave the torch binding out")
    a = ap.parse_args(argv)
    extra = ["-Xptxas", "-v"] if a.ptxas_info else []
    print(build(verbose=a.verbose or a.ptxas_info, force=a.force, extra=extra, binding=not a.no_binding))
    return 0


if __name__ == "__main__":
    sys.exit(main())
