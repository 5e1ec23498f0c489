"""In-tree build of libswiattn.so for sm_103a (GB300), and of the compiled part of the
Python binding.

Each CUDA translation unit is compiled in parallel with nvcc, then linked into
``libswiattn.so`` next to this file.  The CUDA runtime is linked statically and
the driver is reached through cudaGetDriverEntryPointByVersion, so the library
loads on machines without a GPU driver (its entry points then fail with
SWIATTN_ECUDA).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libswiattn.so")
BINDING = os.path.join(PKG, "_binding.so")
TORCH = os.path.join(BUILD, "torch_version")   # what the binding was compiled against

SOURCES = ["swiattn_api.cu", "route.cu", "schedule.cu", "attn_prefill.cu", "attn_simt.cu", "decode.cu",
           "bwd_schedule.cu", "attn_bwd.cu", "bwd_simt.cu", "attn_dual.cu", "rope.cu",
           "decode_e4m3.cu", "paging.cu", "decode_tree.cu",
           "decode_tree_tc.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libswiattn")
    return cand


_BINDING_SOURCE = "binding.cpp"


def _fresh(made: str, sources) -> bool:
    """Whether `made` is there and no older than its sources in csrc and the header."""
    paths = [os.path.join(CSRC, f) for f in sources] + [os.path.join(INCLUDE, "swiattn.h")]
    return os.path.exists(made) and os.path.getmtime(made) >= max(os.path.getmtime(p) for p in paths)


def _build_binding() -> None:
    """csrc/binding.cpp against the installed PyTorch, whose own libraries are loaded before it."""
    import torch
    if os.path.exists(TORCH):   # until the new one is in place, none counts as built
        os.remove(TORCH)
    root = os.path.dirname(torch.__file__)
    lib = os.path.join(root, "lib")
    tmp = BINDING + f".{os.getpid()}.tmp"
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *(f"-I{d}" for d in (INCLUDE, os.path.join(root, "include"),
                                os.path.join(root, "include", "torch", "csrc", "api", "include"),
                                os.path.join(cuda, "include"), sysconfig.get_path("include"))),
           os.path.join(CSRC, _BINDING_SOURCE), "-o", tmp, f"-L{lib}", "-ltorch_python", "-ltorch_cpu",
           "-lc10", "-lc10_cuda"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, BINDING)
    with open(TORCH, "w") as f:
        f.write(_against())


def _against() -> str:
    import torch
    return f"PyTorch {torch.__version__}, Python {sysconfig.get_python_version()}"


def same_torch() -> bool:
    """Whether the binding was compiled against the installed PyTorch (and Python)."""
    try:
        with open(TORCH) as f:
            return f.read() == _against()
    except OSError:
        return False


def _try_binding() -> None:
    """Its calls have a form in Python, so that a machine without a C++ compiler or Python's headers
    does without."""
    try:
        _build_binding()
    except (RuntimeError, OSError) as e:
        warnings.warn(f"the compiled binding was not built: {e}", RuntimeWarning, stacklevel=2)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile (if stale) and return the path of libswiattn.so."""
    binding = force or not (_fresh(BINDING, [_BINDING_SOURCE]) and same_torch())
    library = force or not _fresh(LIB, [f for f in os.listdir(CSRC) if f != _BINDING_SOURCE])
    if not binding and not library:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    if not library:
        _try_binding()
        return LIB
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
        if verbose or ptxas_info:
            print(res.stdout + res.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        beside = ex.submit(_try_binding) if binding else None
        objs = list(ex.map(compile_one, SOURCES))
        if beside:
            beside.result()
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
