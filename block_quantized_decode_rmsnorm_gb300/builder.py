"""Build libqgemv.so in-tree with nvcc for sm_103a.

Each .cu under csrc/ is compiled in parallel to an object in _build/, then the
objects are linked into ``libqgemv.so`` next to this file.  csrc/qg_torch.cpp, the
native front end of the 8-bit floating point calls for torch tensors, becomes
``_qg_torch.so`` beside it (the library itself stays free of torch).  Rebuilds only
when a source, header, flag or the torch version changed.  No cmake, no torch
extension machinery.
"""

from __future__ import annotations

import hashlib
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libqgemv.so")
FRONT_SRC = os.path.join(CSRC, "qg_torch.cpp")
FRONT = os.path.join(HERE, "_qg_torch.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              f"-I{INCLUDE}"]


def _nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand) and not shutil.which(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libqgemv.so")
    return cand


def _torch_dir() -> str | None:
    """Where torch is installed (not imported here); None without it."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _compile_front(torch_dir: str, nvcc: str) -> str:
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    obj = os.path.join(BUILD, "qg_torch.o")
    inc = [INCLUDE, os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    r = subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden",
                        *[f"-I{d}" for d in inc], "-c", FRONT_SRC, "-o", obj], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on qg_torch.cpp:\n{r.stderr}")
    return obj


def _link_front(obj: str, torch_dir: str) -> None:
    lib = os.path.join(torch_dir, "lib")
    tmp = FRONT + f".tmp{os.getpid()}"
    r = subprocess.run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, f"-L{HERE}", "-lqgemv", f"-L{lib}",
                        "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python",
                        "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, FRONT)


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return sorted(hs)


def _digest(paths, extra=""):
    h = hashlib.sha256(extra.encode())
    for p in paths:
        h.update(p.encode())
        with open(p, "rb") as f:
            h.update(f.read())
    return h.hexdigest()


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libqgemv.so (and _qg_torch.so); returns the library's path."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    torch_dir = _torch_dir()
    flags = " ".join(ARCH + NVCC_FLAGS)
    if torch_dir:
        flags += " torch " + importlib.metadata.version("torch")
    digest = _digest(srcs + _headers() + [FRONT_SRC], flags)
    stamp = os.path.join(BUILD, "stamp")
    if not force and os.path.exists(LIB) and (not torch_dir or os.path.exists(FRONT)) and os.path.exists(stamp) \
            and open(stamp).read() == digest:
        return LIB
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        front = ex.submit(_compile_front, torch_dir, nvcc) if torch_dir else None
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    if front:
        _link_front(front.result(), torch_dir)
    with open(stamp, "w") as f:
        f.write(digest)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
