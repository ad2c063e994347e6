"""Build libcb.so in-tree with nvcc for sm_103a (GB300).

Each .cu under csrc/ is compiled in parallel to an object under _build/, then
linked into paged_kv_attention_cb_gb300/libcb.so with the static CUDA runtime.
Beside them csrc/torch_binding.cpp becomes the CPython module _cb_torch.so (the
checked calls from Python; host code only, against this machine's torch).
Run as ``python -m paged_kv_attention_cb_gb300.build`` or call ``build()``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libcb.so")
BINDING_PATH = os.path.join(PKG, "_cb_torch.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
          "--expt-relaxed-constexpr", "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: libcb needs the CUDA toolkit to build")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def _digest(paths, extra=""):
    h = hashlib.sha256(extra.encode())
    for p in paths:
        h.update(p.encode())
        with open(p, "rb") as f:
            h.update(f.read())
    return h.hexdigest()


def _compile(src: str, hdr_digest: str, verbose: bool) -> str:
    base = os.path.splitext(os.path.basename(src))[0]
    obj = os.path.join(BUILD_DIR, base + ".o")
    stamp = obj + ".sha"
    dig = _digest([src], hdr_digest + " ".join(CFLAGS + ARCH))
    if os.path.exists(obj) and os.path.exists(stamp) and open(stamp).read() == dig:
        return obj
    cmd = [nvcc(), *ARCH, *CFLAGS, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
    if verbose and res.stderr.strip():
        print(res.stderr, file=sys.stderr)
    with open(stamp, "w") as f:
        f.write(dig)
    return obj


def _build_binding(hdr_digest: str, verbose: bool) -> None:
    """csrc/torch_binding.cpp -> _cb_torch.so, against this machine's torch."""
    import torch

    src = os.path.join(CSRC, "torch_binding.cpp")
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I" + INCLUDE, "-I" + inc, "-I" + os.path.join(inc, "torch", "csrc", "api", "include"),
           "-I" + cuda, "-I" + sysconfig.get_paths()["include"], src]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    link = ["-L" + libs, "-Wl,-rpath," + libs, "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    stamp = BINDING_PATH + ".sha"
    dig = _digest([src], hdr_digest + " ".join(cmd + link) + torch.__version__)
    if os.path.exists(BINDING_PATH) and os.path.exists(stamp) and open(stamp).read() == dig:
        return
    tmp = BINDING_PATH + ".tmp"
    if verbose:
        print(" ".join([*cmd, "-o", tmp, *link]), flush=True)
    res = subprocess.run([*cmd, "-o", tmp, *link], capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {src}:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, BINDING_PATH)
    with open(stamp, "w") as f:
        f.write(dig)


def build(verbose: bool = False, force: bool = False) -> str:
    """Compile and link libcb.so and _cb_torch.so; returns libcb's path. Incremental on source
    hashes."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    if force:
        for p in glob.glob(os.path.join(BUILD_DIR, "*")):
            os.remove(p)
    hdr = _digest(_headers())
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_build_binding, hdr, verbose)
        objs = list(ex.map(lambda s: _compile(s, hdr, verbose), srcs))
        binding.result()
    link_stamp = LIB_PATH + ".sha"
    dig = _digest(objs)
    if os.path.exists(LIB_PATH) and os.path.exists(link_stamp) and open(link_stamp).read() == dig:
        return LIB_PATH
    tmp = LIB_PATH + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs, "-ldl", "-lpthread",
           "-lrt"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB_PATH)
    with open(link_stamp, "w") as f:
        f.write(dig)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True, force="--force" in sys.argv))
