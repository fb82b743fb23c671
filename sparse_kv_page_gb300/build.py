"""Builds the in-tree CUDA library ``liblocks_gb300.so`` (sm_103a only).

Each ``csrc/*.cu`` translation unit is compiled in parallel with nvcc, then
linked into one shared library exporting the C ABI of ``include/locks.h``,
``include/locks_cache.h`` and ``include/locks_pool.h``. ``csrc/marshal.cpp`` becomes the extension module ``_marshal``,
the argument checks of the cache operators' Python binding (g++, torch's headers).
Run as ``python -m sparse_kv_page_gb300.build`` or through
``__graft_entry__.build()``.
"""

from __future__ import annotations

import concurrent.futures
import glob
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig
from typing import List

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_NAME = "liblocks_gb300.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
MARSHAL_SRC = os.path.join(CSRC, "marshal.cpp")
MARSHAL_PATH = os.path.join(PKG, "_marshal.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    return os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"


def _flags() -> List[str]:
    return ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
            "--expt-relaxed-constexpr", f"-I{INCLUDE}", "-DLOCKS_BUILD"] + ARCH


def _sources() -> List[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _fingerprint() -> str:
    h = hashlib.sha256()
    files = _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + sorted(
        glob.glob(os.path.join(CSRC, "*.h"))) + sorted(glob.glob(os.path.join(INCLUDE, "*.h"))) + [MARSHAL_SRC]
    for f in files:
        with open(f, "rb") as fh:
            h.update(f.encode() + b"\0" + fh.read())
    h.update(" ".join(_flags()).encode())
    h.update(os.uname().machine.encode())
    h.update(torch.__version__.encode())          # _marshal is compiled against it
    return h.hexdigest()


def source_hash(names) -> str:
    """SHA-256 (hex) of the named files under csrc/ or include/, in the order given:
    identifies a kernel's source independently of the machine that builds it."""
    h = hashlib.sha256()
    for n in names:
        path = os.path.join(CSRC, n)
        if not os.path.exists(path):
            path = os.path.join(INCLUDE, n)
        with open(path, "rb") as fh:
            h.update(n.encode() + b"\0" + fh.read())
    return h.hexdigest()


def _build_marshal() -> None:
    """Compile csrc/marshal.cpp against this interpreter and its torch."""
    root = os.path.dirname(os.path.abspath(torch.__file__))
    lib = os.path.join(root, "lib")
    tmp = MARSHAL_PATH + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-isystem", os.path.join(root, "include"), "-isystem", os.path.join(root, "include/torch/csrc/api/include"),
           "-I", sysconfig.get_paths()["include"], MARSHAL_SRC, "-o", tmp, f"-L{lib}", "-ltorch_python", "-ltorch_cpu",
           "-ltorch", "-lc10", f"-Wl,-rpath,{lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {MARSHAL_SRC}:\n{r.stderr}")
    os.replace(tmp, MARSHAL_PATH)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile (if sources changed) and return the library path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    stamp = os.path.join(BUILD_DIR, "stamp")
    fp = _fingerprint()
    if not force and os.path.exists(LIB_PATH) and os.path.exists(MARSHAL_PATH) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read().strip() == fp:
                return LIB_PATH
    nvcc = _nvcc()
    flags = _flags() + (["-Xptxas", "-v"] if ptxas_info else [])

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc] + flags + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stderr)
        return obj

    srcs = _sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        marshal = ex.submit(_build_marshal)
        objs = list(ex.map(compile_one, srcs))
        marshal.result()
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcudart_static", "-lrt", "-ldl", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    with open(stamp, "w") as f:
        f.write(fp)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
