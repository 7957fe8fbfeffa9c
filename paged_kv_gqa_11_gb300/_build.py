"""Build libpa.so (the C-ABI library) in-tree with nvcc for sm_103a, and the
Python module over it.

Translation units compile in parallel; the CUDA runtime is linked shared so
that the library and PyTorch use one runtime (one current device, one set of
streams) in the same process.  The library has no torch in it: it is linked
whether or not the module compiles, and without torch it is all that is built.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(OUT_DIR, "libpa.so")
CALLS_PATH = os.path.join(OUT_DIR, "pa_calls.so")  # the Python module over it (csrc/pa_calls.cpp)
CALLS_TAG = CALLS_PATH + ".tag"  # the Python and torch it was built against
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
TYPES = {"f16": 1, "q4_0": 2, "q8_0": 8}  # pa_type numbers
# (source, object name, extra defines): the split-decode and shared-prefix
# kernels are one source each, compiled once per (K, V) format pair.
UNITS = [("pa_pool.cpp", "pa_pool", []), ("pa_append.cu", "pa_append", []), ("pa_decode.cu", "pa_decode", []),
         ("pa_rope.cu", "pa_rope", []), ("pa_prefix.cu", "pa_prefix", [])]
UNITS += [("pa_decode_kern.cu", f"pa_decode_kern_{k}_{v}", [f"-DPA_KT={TYPES[k]}", f"-DPA_VT={TYPES[v]}"])
          for k in TYPES for v in TYPES]
UNITS += [("pa_prefix_kern.cu", f"pa_prefix_kern_{k}_{v}", [f"-DPA_KT={TYPES[k]}", f"-DPA_VT={TYPES[v]}"])
          for k in TYPES for v in TYPES]


def _cuda_home() -> str:
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    return os.environ.get("CUDA_HOME", "/usr/local/cuda")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "pa.h"))
    files.append(os.path.abspath(__file__))
    return files


def _torch():
    try:
        import torch
    except ImportError:
        return None
    return torch


def _calls_tag() -> str:
    return f"{sysconfig.get_config_var('SOABI')} torch {_torch().__version__}"


def up_to_date() -> bool:
    built = [LIB_PATH]
    if _torch() is not None:
        built += [CALLS_PATH, CALLS_TAG]
    if not all(os.path.exists(f) for f in built):
        return False
    t = min(os.path.getmtime(f) for f in built)
    if not all(os.path.getmtime(f) <= t for f in _inputs()):
        return False
    if len(built) == 1:
        return True
    with open(CALLS_TAG) as f:
        return f.read() == _calls_tag()


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB_PATH
    cuda = _cuda_home()
    nvcc = os.path.join(cuda, "bin", "nvcc")
    obj_dir = os.path.join(OUT_DIR, "obj")
    os.makedirs(obj_dir, exist_ok=True)
    procs = []
    objs = []
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    torch = _torch()
    calls_obj = os.path.join(obj_dir, "pa_calls.o")
    calls = _calls_compile(torch, cuda, calls_obj) if torch else None
    for src, name, defs in UNITS:
        path = os.path.join(CSRC, src)
        obj = os.path.join(obj_dir, name + ".o")
        objs.append(obj)
        if src.endswith(".cu"):
            cmd = [nvcc, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                   "-I", INCLUDE, "-I", CSRC, *defs, "-c", path, "-o", obj]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
        else:
            cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE, "-I", os.path.join(cuda, "include"),
                   "-c", path, "-o", obj]
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = [" ".join(cmd) for cmd, p in procs if not _finished(p, verbose)]
    calls_ok = calls is None or _finished(calls[1], verbose)
    if failed:
        raise RuntimeError("libpa build failed:\n" + "\n".join(failed))
    link = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-Xcompiler", "-fPIC",
            "-Xlinker", "-rpath", "-Xlinker", os.path.join(cuda, "lib64"), *objs, "-o", tmp]
    subprocess.run(link, check=True)
    os.replace(tmp, LIB_PATH)
    if not calls_ok:
        if os.path.exists(CALLS_PATH):  # made for another libpa
            os.remove(CALLS_PATH)
        raise RuntimeError("pa_calls build failed (libpa is built):\n" + " ".join(calls[0]))
    if calls is not None:
        lib = os.path.join(os.path.dirname(torch.__file__), "lib")
        tmp = CALLS_PATH + f".tmp{os.getpid()}"
        subprocess.run(["g++", "-shared", calls_obj, "-o", tmp, "-L", OUT_DIR, "-l:libpa.so", "-L", lib, "-ltorch_python", "-ltorch",
                        "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"], check=True)
        os.replace(tmp, CALLS_PATH)
        with open(CALLS_TAG, "w") as f:
            f.write(_calls_tag())
    return LIB_PATH


def _finished(p, verbose: bool) -> bool:
    out, _ = p.communicate()
    if verbose or p.returncode:
        print(out.decode(errors="replace"))
    return p.returncode == 0


def _calls_compile(torch, cuda: str, obj: str):
    """The Python module's compilation, against torch's own headers."""
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    abi = int(getattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", True))
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={abi}", "-I", INCLUDE, "-isystem", inc, "-isystem",
           os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", sysconfig.get_paths()["include"], "-isystem",
           os.path.join(cuda, "include"), "-c", os.path.join(CSRC, "pa_calls.cpp"), "-o", obj]
    return cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)


if __name__ == "__main__":
    print(build(force=True, verbose=True))
