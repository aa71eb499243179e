"""Builds ``libfa2_gb300.so`` from ``csrc/`` with nvcc for sm_103a only.

Each translation unit compiles in its own nvcc process (in parallel); the
objects are linked into one shared library with the CUDA runtime linked
statically.  Beside it ``_fa2_torch.so``, the CPython extension that reads the
serving calls' torch tensors (``csrc/torch_args.cpp``), is compiled with g++
against the installed torch; without a torch only the library is built, which
needs none.  Either is rebuilt only when a source or header of its own is newer,
the extension also when it was compiled against another torch or Python (or when
``force=True``).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libfa2_gb300.so")
TORCH_LIB = os.path.join(HERE, "_fa2_torch.so")
TORCH_SRC = os.path.join(CSRC, "torch_args.cpp")
TORCH_STAMP = os.path.join(BUILD_DIR, "_fa2_torch.torch")  # the torch and Python it was compiled against

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
         "--expt-relaxed-constexpr", "-Xcompiler", "-Wall"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _torch_dir():
    """Where the installed torch lies (not imported for it); None without one."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _torch_stamp(torch: str) -> str:
    """What an extension compiled now belongs to: it reads torch's objects at this version's offsets."""
    version = os.path.join(torch, "version.py")
    text = open(version).read() if os.path.exists(version) else ""
    return f"{torch}\n{sys.version}\n{text}"


def _build_extension(nvcc: str, torch: str) -> str:
    """Compile csrc/torch_args.cpp against torch; returns the compiler's output."""
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    tmp = TORCH_LIB + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", TORCH_SRC, "-o", tmp, "-I", INCLUDE,
           "-isystem", os.path.join(torch, "include"), "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_path("include"), "-isystem", os.path.join(cuda, "include"),
           "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {TORCH_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, TORCH_LIB)
    with open(TORCH_STAMP, "w") as f:
        f.write(_torch_stamp(torch))
    return r.stdout + r.stderr


def _older(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in deps)


def _library_stale() -> bool:
    return _older(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def _extension_stale(torch: str) -> bool:
    if _older(TORCH_LIB, [TORCH_SRC] + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]):
        return True
    return not os.path.exists(TORCH_STAMP) or open(TORCH_STAMP).read() != _torch_stamp(torch)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile what is stale: the library, and with a torch installed its extension; returns the library's path."""
    torch = _torch_dir()
    if torch is None:
        print("torch is not installed: _fa2_torch.so, through which the serving calls take its tensors, is not built", file=sys.stderr)
    library, extension = force or _library_stale(), torch is not None and (force or _extension_stale(torch))
    if not library and not extension:
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        beside = ex.submit(_build_extension, nvcc, torch) if extension else None
        log = _build_library(nvcc, ["-Xptxas", "-v"] if ptxas_info else []) if library else ""
        log += beside.result() if beside else ""
    if (verbose or ptxas_info) and log.strip():
        sys.stdout.write(log)
    return LIB


def _build_library(nvcc: str, extra) -> str:
    """Compile every CUDA source and link the library; returns the compiler's output."""
    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        results = list(ex.map(compile_one, sources()))
    objs = [o for o, _ in results]
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return "".join(log for _, log in results)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas-info" in sys.argv))
