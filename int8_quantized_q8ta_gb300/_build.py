"""Build libq8ta.so (the C-ABI library of include/q8ta.h) in-tree with nvcc, and
_torch_calls.so (csrc/torch_calls.cpp, a Python module that calls it with torch's
tensors) beside it with g++.

Each CUDA source is compiled for sm_103a only (explicit
``-gencode arch=compute_103a,code=sm_103a``; tcgen05 needs the ``a`` target),
in parallel, then linked into ``int8_quantized_q8ta_gb300/libq8ta.so``.
Host code has no architecture-specific flags, so the same sources build on
x86-64 and aarch64 hosts.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ_DIR = os.path.join(PKG, "_objs")
LIB = os.path.join(PKG, "libq8ta.so")
CALLS = os.path.join(PKG, "_torch_calls.so")
CALLS_SRC = os.path.join(CSRC, "torch_calls.cpp")
CALLS_KEY = os.path.join(OBJ_DIR, "torch_calls.key")   # the torch that CALLS was built against

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the q8ta CUDA library cannot be built")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + [CALLS_SRC] + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")) + \
        [os.path.abspath(__file__)]


def _torch_key() -> str:
    """Which torch and Python a module built now would be of (torch is found, not
    imported)."""
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None:
        return ""
    with open(os.path.join(os.path.dirname(spec.origin), "version.py")) as f:
        version = f.read()
    return "\n".join([spec.origin, str(sysconfig.get_config_var("SOABI")), version])


def _built_key() -> str:
    if not os.path.exists(CALLS_KEY):
        return ""
    with open(CALLS_KEY) as f:
        return f.read()


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(CALLS)) or _built_key() != _torch_key():
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(CALLS))
    return all(os.path.getmtime(d) <= t for d in _deps())


def _compile_calls() -> str:
    """The object of the Python module (the headers are torch's own, those of the
    torch that will import it)."""
    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    obj = os.path.join(OBJ_DIR, "torch_calls.o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-c", CALLS_SRC, "-o", obj,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE]
    for path in (os.path.join(root, "include"),
                 os.path.join(root, "include", "torch", "csrc", "api", "include"),
                 sysconfig.get_paths()["include"], os.path.join(cuda, "include")):
        cmd += ["-isystem", path]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on torch_calls.cpp:\n{r.stderr}")
    return obj


def _link_calls(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(os.path.abspath(torch.__file__)), "lib")
    tmp = CALLS + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", PKG, "-l:libq8ta.so", "-Wl,-rpath,$ORIGIN", "-L",
           libs, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", f"-Wl,-rpath,{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ link failed:\n{r.stderr}")
    os.replace(tmp, CALLS)
    with open(CALLS_KEY, "w") as f:
        f.write(_torch_key())


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile and link the library if any source is newer.  Returns its path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(OBJ_DIR, exist_ok=True)
    cc = nvcc()
    flags = NVCC_FLAGS + list(extra_flags or [])
    if verbose:
        flags = flags + ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(OBJ_DIR, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        calls = ex.submit(_compile_calls)
        results = list(ex.map(compile_one, _sources()))
        calls_obj = calls.result()
    if verbose:
        for _, err in results:
            if err.strip():
                print(err)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_calls(calls_obj)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
