"""Build libmxq.so in-tree for sm_103a.

Each CUDA translation unit is compiled by nvcc in parallel with
``-gencode arch=compute_103a,code=sm_103a``, the C-ABI layer by the host
compiler, and the objects are linked into ``libmxq.so`` next to this file.
``mxq_fastcall``, the binding's quick way into it for common calls, is built beside
it against the installed torch, and named after torch's and Python's versions;
where there is none for them (no torch or Python headers) the binding makes those
calls through ctypes like all others.
A build is skipped when the library is newer than every source and header; a missing
or older ``mxq_fastcall`` for the installed torch is then built alone.  A new library
takes away the modules that were built beside the old one, for whatever torch.
"""

from __future__ import annotations

import concurrent.futures as cf
import importlib.machinery
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libmxq.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CU_SOURCES = ["quant.cu", "misc.cu", "bmm.cu", "linear_noalloc.cu", "kv_insert.cu", "kv4.cu",
              "attn.cu", "norm.cu", "route.cu", "w4.cu"]
CXX_SOURCES = ["api.cpp"]


def fastcall_path(torch_version) -> str:
    """Where the quick way in for this torch and this Python lies."""
    return os.path.join(HERE, f"mxq_fastcall-{torch_version}{importlib.machinery.EXTENSION_SUFFIXES[0]}")


def cuda_home() -> str:
    for cand in (os.environ.get("CUDA_HOME"), os.environ.get("CUDA_PATH"), "/usr/local/cuda"):
        if cand and os.path.exists(os.path.join(cand, "bin", "nvcc")):
            return cand
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    raise RuntimeError("nvcc not found (set CUDA_HOME)")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "mxq.h"))
    files.append(os.path.abspath(__file__))
    return files


def _current(path) -> bool:
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def up_to_date() -> bool:
    return _current(LIB_PATH)


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"command failed ({r.returncode}): {' '.join(cmd)}\n{r.stdout}")
    return r.stdout


_tried = set()  # modules that this process could not build


def _fastcall_wanted(anew):
    """Where the quick way in for the installed torch has to be built (`anew`: though it is current), or None."""
    try:
        import torch
    except ImportError:
        return None
    path = fastcall_path(torch.__version__)
    return None if path in _tried or (not anew and _current(path)) else path


def _includes():
    return ["-I", INCLUDE, "-I", CSRC, "-I", os.path.join(cuda_home(), "include")]


def _compile_fastcall(path, verbose):
    """Compile mxq_fastcall beside its place; a failure leaves it out, with a message.  Returns whether it is there."""
    try:
        import torch

        at = os.path.dirname(torch.__file__)
        _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-Wall", "-shared",
              f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *_includes(),
              "-isystem", os.path.join(at, "include"),
              "-isystem", os.path.join(at, "include", "torch", "csrc", "api", "include"),
              "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, "fastcall.cpp"), "-o", path + ".tmp",
              "-L", os.path.join(at, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"], verbose)
    except (RuntimeError, OSError) as e:
        print(f"mxq_fastcall not built: {e}", file=sys.stderr, flush=True)
        _tried.add(path)
        return False
    return True


def _remove_fastcalls(but=None) -> None:
    """Take away the modules for every torch and Python (but for files beginning with `but`)."""
    for f in os.listdir(HERE):
        if f.startswith("mxq_fastcall-") and not (but and f.startswith(os.path.basename(but))):
            os.remove(os.path.join(HERE, f))


def build(verbose: bool = False, force: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link libmxq.so; returns its path."""
    if force:
        _tried.clear()
    library = force or not up_to_date()
    fast = _fastcall_wanted(anew=library)
    if not library:
        if fast is not None:
            if os.path.exists(fast):  # an older one, of other arguments perhaps
                os.remove(fast)
            if _compile_fastcall(fast, verbose):
                os.replace(fast + ".tmp", fast)
        return LIB_PATH
    home = cuda_home()
    nvcc = os.path.join(home, "bin", "nvcc")
    cxx = os.environ.get("CXX", "g++")
    inc = _includes()
    os.makedirs(BUILD_DIR, exist_ok=True)
    jobs = []
    for src in CU_SOURCES:
        obj = os.path.join(BUILD_DIR, src + ".o")
        cmd = [nvcc, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
               "--expt-relaxed-constexpr", *inc, "-c", os.path.join(CSRC, src), "-o", obj]
        if ptxas_info:
            cmd.insert(1, "-Xptxas=-v")
        jobs.append((cmd, obj))
    for src in CXX_SOURCES:
        obj = os.path.join(BUILD_DIR, src + ".o")
        cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-Wall", *inc, "-c", os.path.join(CSRC, src),
               "-o", obj]
        jobs.append((cmd, obj))
    outputs = []
    with cf.ThreadPoolExecutor(max_workers=len(jobs) + 1) as ex:
        made = fast and ex.submit(_compile_fastcall, fast, verbose)
        for out in ex.map(lambda j: _run(j[0], verbose), jobs):
            outputs.append(out)
        made = made and made.result()
    if ptxas_info:
        print("\n".join(outputs))
    tmp = LIB_PATH + ".tmp"
    _run([nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *[o for _, o in jobs],
          "-L", os.path.join(home, "lib64")], verbose)
    # The modules pass their arguments by the old library's header.
    _remove_fastcalls(but=fast + ".tmp" if made else None)
    os.replace(tmp, LIB_PATH)
    if made:
        os.replace(fast + ".tmp", fast)
    return LIB_PATH


if __name__ == "__main__":
    build(verbose=True, force="--force" in sys.argv, ptxas_info="--ptxas-info" in sys.argv)
    print(LIB_PATH)
