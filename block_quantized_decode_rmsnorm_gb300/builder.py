"""Build libqgemv.so in-tree with nvcc for sm_103a.

Each .cu under csrc/ is compiled in parallel to an object in _build/, then the
objects are linked into ``libqgemv.so`` next to this file.  csrc/qg_torch.cpp, the
native front end of the 8-bit floating point calls for torch tensors, becomes the
extension module ``_qg_torch`` beside it, where torch is installed with CUDA (the
library itself needs nvcc alone).  Each is rebuilt only when what it is made from
changed: sources, headers and flags; for the front end the interpreter, torch and the
compiler as well.  No cmake, no torch extension machinery.
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
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libqgemv.so")
FRONT_SRC = os.path.join(CSRC, "qg_torch.cpp")
FRONT = os.path.join(HERE, "_qg_torch" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))  # this interpreter's

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              f"-I{INCLUDE}"]


def _nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand) and not shutil.which(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libqgemv.so")
    return cand


def _torch_dir() -> str | None:
    """Where torch is installed with CUDA (not imported here); None without."""
    spec = importlib.util.find_spec("torch")
    d = os.path.dirname(spec.origin) if spec and spec.origin else None
    return d if d and os.path.exists(os.path.join(d, "lib", "libc10_cuda.so")) else None


def _cxx() -> str:
    return os.environ.get("CXX", "g++")


def _front_digest() -> str:
    return _digest([FRONT_SRC, *_headers()], " ".join(
        [sys.implementation.cache_tag or "", FRONT, importlib.metadata.version("torch"), _cxx()]))


def _compile_front(torch_dir: str, nvcc: str) -> None:
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    lib = os.path.join(torch_dir, "lib")
    inc = [INCLUDE, os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    tmp = FRONT + f".tmp{os.getpid()}"
    try:
        r = subprocess.run([_cxx(), "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden", *[f"-I{d}" for d in inc], "-shared",
                            "-o", tmp, FRONT_SRC, f"-L{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python",
                            f"-Wl,-rpath,{lib}"],
                           capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError(f"{_cxx()}: {e}") from e
    if r.returncode != 0:
        raise RuntimeError(f"{_cxx()} failed on qg_torch.cpp:\n{r.stderr}")
    os.replace(tmp, FRONT)


def _current(stamp: str, digest: str, made: str) -> bool:
    if not os.path.exists(made) or not os.path.exists(stamp):
        return False
    with open(stamp) as f:
        return f.read() == digest


def _build_front(torch_dir: str, force: bool) -> None:
    stamp, digest = os.path.join(BUILD, "stamp_" + os.path.basename(FRONT)), _front_digest()
    if not force and _current(stamp, digest, FRONT):
        return
    if os.path.exists(FRONT):  # an older one would be taken for this one's
        os.remove(FRONT)
    _compile_front(torch_dir, _nvcc())
    with open(stamp, "w") as f:
        f.write(digest)


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


def _build_library(force: bool, verbose: bool) -> None:
    srcs = _sources()
    digest = _digest(srcs + _headers(), " ".join(ARCH + NVCC_FLAGS))
    stamp = os.path.join(BUILD, "stamp")
    if not force and _current(stamp, digest, LIB):
        return
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

    with ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    with open(stamp, "w") as f:
        f.write(digest)


def build(force: bool = False, verbose: bool = False, strict: bool = False) -> str:
    """Compile and link libqgemv.so, and the torch front end where torch has CUDA; returns
    the library's path.  A front end that cannot be built is a warning, as the library and
    what needs no more than it are there (the 8-bit floating point calls for torch tensors
    then raise); with ``strict`` it is an error."""
    os.makedirs(BUILD, exist_ok=True)
    torch_dir = _torch_dir()
    with ThreadPoolExecutor(max_workers=1) as ex:  # it is linked to torch alone: at the same time
        front = ex.submit(_build_front, torch_dir, force) if torch_dir else None
        _build_library(force, verbose)
    if front:
        try:
            front.result()
        except Exception as e:  # whatever it is, the library is there
            if strict:
                raise
            warnings.warn(f"the torch front end was not built: {e}", RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, strict=True))
