"""Build ``libgemmepi.so`` in-tree with nvcc for sm_103a.

Each translation unit under ``csrc/`` is compiled in parallel (``-gencode
arch=compute_103a,code=sm_103a -lineinfo -O3``), with the CUDA runtime linked statically,
so the library needs only the NVIDIA driver at run time; ``-Xptxas -v`` register and
shared-memory reports are kept in ``_build/ptxas.log``.

    python -m activation_epilogue_gb300.build [--force]
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libgemmepi.so")
SOURCES = ["api.cu", "host_exec.cu", "ffn_api.cu", "layernorm_api.cu", "gemm_pair.cu",
           "gemm_pair_fp8.cu", "gemm_block_square.cu", "gemm_block_rows.cu", "gemm_block_swapped.cu",
           "gemm_rowtile.cu", "gemm_swapped.cu", "gemm_fwd_bias.cu", "gemm_fwd_relu.cu",
           "gemm_fwd_gelu.cu", "gemm_fwd_relu_aux.cu", "gemm_fwd_residual.cu",
           "gemm_smallm.cu", "ffn_onchip.cu", "elementwise.cu", "layernorm.cu",
           "sublayer_api.cu", "rmsnorm.cu", "layernorm_train.cu", "quantize.cu", "w4.cu",
           "w4_stream.cu", "w4_tensor.cu", "dropout.cu"]
# The binding's marshalling in C++.  It needs the headers of Python and of a torch built with CUDA, and
# that torch's libraries; without them the binding goes through ctypes.  It reaches into torch's tensors,
# so it belongs to one torch, which the stamp beside it names.
FASTCALL = os.path.join(PKG, "_fastcall.so")
FASTCALL_SRC = os.path.join(CSRC, "fastcall.cpp")
FASTCALL_STAMP = os.path.join(BUILD, "fastcall.torch")
FASTCALL_LIBS = ("torch_python", "torch_cpu", "c10", "c10_cuda")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "gemm_epi.h"))
    return [f for f in files if os.path.isfile(f)]


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in _deps() + [__file__])


def _torch_dir() -> str | None:
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec and spec.submodule_search_locations else None


def _fastcall_paths() -> tuple[list[str], str] | None:
    """(include folders, torch's library folder), or None where something that it needs is missing."""
    torch_dir = _torch_dir()
    if torch_dir is None:
        return None
    nvcc = _nvcc()
    includes = [sysconfig.get_path("include"), os.path.join(torch_dir, "include"),
                os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
                os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")]
    libdir = os.path.join(torch_dir, "lib")
    needed = [os.path.join(includes[0], "Python.h"),
              os.path.join(includes[1], "torch", "csrc", "autograd", "python_variable.h"),
              os.path.join(includes[1], "c10", "cuda", "CUDAStream.h"),
              os.path.join(includes[3], "cuda_runtime_api.h"),
              *(os.path.join(libdir, f"lib{name}.so") for name in FASTCALL_LIBS)]
    if not all(os.path.exists(f) for f in needed):
        return None
    return includes, libdir


def _fastcall_torch() -> str:
    """The torch and the Python that the marshalling is built for."""
    torch_dir = _torch_dir()
    try:
        with open(os.path.join(torch_dir, "version.py")) as fh:
            version = fh.read()
    except OSError:
        version = ""
    return f"{sys.version}\n{torch_dir}\n{version}"


def _fastcall_current() -> bool:
    """The marshalling is there, newer than its sources, and of this torch."""
    if not os.path.exists(FASTCALL) or not os.path.exists(FASTCALL_STAMP):
        return False
    t = os.path.getmtime(FASTCALL)
    if any(os.path.getmtime(f) > t for f in (FASTCALL_SRC, os.path.join(INCLUDE, "gemm_epi.h"), __file__)):
        return False
    with open(FASTCALL_STAMP) as fh:
        return fh.read() == _fastcall_torch()


def _fastcall_stale() -> bool:
    """It has to be built, or taken away where it is another torch's and cannot be built for this one."""
    return not _fastcall_current() and (os.path.exists(FASTCALL) or _fastcall_paths() is not None)


def _compile_fastcall() -> None:
    paths = _fastcall_paths()
    if paths is None:
        if os.path.exists(FASTCALL):
            os.remove(FASTCALL)
        return
    includes, libdir = paths
    tmp = FASTCALL + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE]
    for folder in includes:
        cmd += ["-isystem", folder]
    cmd += [FASTCALL_SRC, "-L", libdir, *(f"-l{name}" for name in FASTCALL_LIBS),
            f"-Wl,-rpath,{libdir}", "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on fastcall.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, FASTCALL)
    with open(FASTCALL_STAMP, "w") as fh:
        fh.write(_fastcall_torch())


def _compile(nvcc: str, src: str) -> tuple[str, str]:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc, *ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
           "-Xptxas", "-v", "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def build(force: bool = False, verbose: bool = False) -> str:
    library, marshalling = force or _stale(), force or _fastcall_stale()
    if not library and not marshalling:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        fastcall = ex.submit(_compile_fastcall) if marshalling else None
        if library:
            _link(nvcc, list(ex.map(lambda s: _compile(nvcc, s), SOURCES)))
        if fastcall:
            fastcall.result()
    if verbose:
        print(f"built {LIB}")
    return LIB


def _link(nvcc: str, results: list[tuple[str, str]]) -> None:
    with open(os.path.join(BUILD, "ptxas.log"), "w") as fh:
        for src, (_, log) in zip(SOURCES, results):
            fh.write(f"==== {src}\n{log}\n")
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
