"""Builds the CUDA library libgbnorm.so in-tree for sm_103a.

Its translation units (bf16- and E4M3-output forward, forward with staged
parameters, backward, long-row kernels plain, with the fused residual add and
with E4M3 output, the streamed rows, the two-pass path for the longest rows,
host ABI, host-tensor pipeline, the normalisation fused into a tcgen05 GEMM,
dropout, dropout + residual add + norm, and group normalisation) are
compiled in parallel with nvcc and linked into one shared object with the
CUDA runtime linked statically, so the library needs no CUDA library path at
load time.  Beside it a small extension module, gbnorm_torch.so, is compiled
against PyTorch's headers and linked to the library: the tensor side of the
dropout and group-normalisation entry points.  It belongs to one PyTorch and one
Python, which gbnorm_torch.stamp names: for others it is built again, and not
loaded before that.  A PyTorch without CUDA has no tensors for it, so there the
library alone is built.  `python -m memory_bound_normalization_rmsnorm_gb300.builder -v`
also prints ptxas register/spill/shared-memory figures.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "lib")
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libgbnorm.so")
TORCH_LIB = os.path.join(OUT_DIR, "gbnorm_torch.so")
TORCH_STAMP = os.path.join(OUT_DIR, "gbnorm_torch.stamp")
SOURCES = ["fwd.cu", "fwd_fp8.cu", "fwd_gsm.cu", "bwd.cu", "long.cu", "long_resid.cu",
           "long_fp8.cu", "split.cu", "stream.cu", "api.cu", "host.cu", "gemm.cu", "dropout.cu",
           "drop_add.cu", "group_fwd.cu", "group_bwd.cu", "group_ring.cu",
           "group.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc():
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgbnorm")
    return cand


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "gbnorm.h"))
    files.append(os.path.abspath(__file__))
    return files


def _fresh(path):
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(f) <= t for f in _deps())


def torch_stamp() -> str:
    """The PyTorch and Python that an extension module built now is for."""
    import torch

    return (f"torch {torch.__version__} cxx11abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)} "
            f"python {sysconfig.get_config_var('SOABI')}\n")


def torch_lib_stamp() -> str:
    """The PyTorch and Python that the present extension module is for."""
    if not os.path.exists(TORCH_STAMP):
        return ""
    with open(TORCH_STAMP) as f:
        return f.read()


def _torch_has_cuda():
    import torch

    return torch.version.cuda is not None


def _binding_up_to_date():
    if not _torch_has_cuda():
        return True
    return _fresh(TORCH_LIB) and torch_lib_stamp() == torch_stamp()


def up_to_date() -> bool:
    return _fresh(LIB) and _binding_up_to_date()


def _torch_compile():
    """Compiles the tensor binding; returns its object file."""
    import torch

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    obj = os.path.join(BUILD_DIR, "torch_binding.o")
    cmd = ["g++", "-c", os.path.join(CSRC, "torch_binding.cpp"), "-o", obj, "-O2", "-std=c++17",
           "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"),
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on torch_binding.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _torch_link(obj):
    import torch

    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = TORCH_LIB + f".tmp{os.getpid()}"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", OUT_DIR, "-lgbnorm", "-Wl,-rpath,$ORIGIN",
           "-L", libs, "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    # (no stamp while the module changes: a stale one must not vouch for it)
    if os.path.exists(TORCH_STAMP):
        os.remove(TORCH_STAMP)
    os.replace(tmp, TORCH_LIB)
    with open(TORCH_STAMP, "w") as f:
        f.write(torch_stamp())


def build(force: bool = False, verbose: bool = False) -> str:
    library = force or not _fresh(LIB)
    binding = _torch_has_cuda() and (library or not _binding_up_to_date())
    os.makedirs(OUT_DIR, exist_ok=True)
    os.makedirs(BUILD_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(1) as ex:
        obj = ex.submit(_torch_compile) if binding else None
        if library:
            _build_library(verbose)
        if obj:
            _torch_link(obj.result())
    return LIB


def _build_library(verbose):
    nvcc = _nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-I", INCLUDE, "-I", CSRC]
    if verbose:
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [nvcc, "-c", os.path.join(CSRC, src), "-o", obj] + flags
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, "-shared", "-o", tmp] + ARCH + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force=True, verbose="-v" in sys.argv))
