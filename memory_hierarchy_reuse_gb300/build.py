"""Build libmhr_gemm.so (the C-ABI GEMM library) for sm_103a with nvcc.

Each translation unit is compiled in parallel, then linked into a shared
library inside this package directory (the CUDA runtime is linked statically,
so the library needs only the NVIDIA driver at run time). Beside it g++ compiles
the 4-bit tensor-level calls' binding (_torch_binding.so) against the installed
torch, again whenever that is another one; without torch it is left out.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmhr_gemm.so")
SOURCES = ["api.cu", "simt_f32.cu", "tc_gemm.cu", "tc_gemm_1cta.cu", "tc_gemm_pair.cu",
           "tc_prepass.cu", "noalloc.cu", "ladder.cu", "mxfp4_api.cu", "mxfp4_quantize.cu",
           "mxfp4_narrow.cu", "mxfp4_pair.cu", "mxfp4_moe.cu"]
BINDING = os.path.join(PKG, "_torch_binding.so")
BINDING_SOURCE = os.path.join(CSRC, "torch_binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale(target: str, folders: list[str], names: tuple[str, ...]) -> bool:
    """Whether `target` is missing or older than a file of `folders` with one of the endings."""
    if not os.path.exists(target):
        return True
    files = [os.path.join(d, f) for d in folders for f in os.listdir(d) if f.endswith(names)]
    t = os.path.getmtime(target)
    return any(os.path.getmtime(f) > t for f in files + [os.path.abspath(__file__)])


def _torch_root() -> str | None:
    """The folder of the installed torch, found without importing it."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(os.path.abspath(spec.origin)) if spec and spec.origin else None


def _torch_stamp(root: str) -> str:
    """What a binding is compiled against: this interpreter, and torch's place and version."""
    with open(os.path.join(root, "version.py")) as f:
        return f"{sys.version}\n{root}\n{f.read()}"


def _stamp_file() -> str:
    return os.path.join(BUILD_DIR, "torch_binding.stamp")


def _binding_stale(stamp: str) -> bool:
    if _stale(BINDING, [CSRC, INCLUDE], (".cpp", ".h")) or not os.path.exists(_stamp_file()):
        return True
    with open(_stamp_file()) as f:
        return f.read() != stamp


def _build_binding() -> None:
    """The torch binding: host code only, against torch's headers and libraries."""
    import torch

    root = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    lib = os.path.join(root, "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(root, "include"),
           "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(cuda, "include"), "-I", sysconfig.get_paths()["include"],
           "-I", INCLUDE, BINDING_SOURCE, "-o", tmp, "-L", lib, f"-Wl,-rpath,{lib}",
           "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on torch_binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile and link what changed; returns the library's path. The library is linked before an
    error of the binding is raised."""
    root = _torch_root()
    stamp = _torch_stamp(root) if root else ""
    library = force or _stale(LIB, [CSRC, INCLUDE], (".cu", ".cuh", ".h"))
    bind = root is not None and (force or _binding_stale(stamp))
    if library or bind:
        os.makedirs(BUILD_DIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(_build_binding) if bind else None
        if library:
            if not root:
                sys.stderr.write("no torch: libmhr_gemm.so is built without the 4-bit tensor calls\n")
            _build_library(verbose_ptxas)
        if binding:
            binding.result()
            with open(_stamp_file(), "w") as f:
                f.write(stamp)
    return LIB


def _build_library(verbose_ptxas: bool) -> None:
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
                    "-I", INCLUDE, "-I", CSRC]
    if verbose_ptxas or os.environ.get("MHR_PTXAS_VERBOSE"):
        flags += ["-Xptxas", "-v"]
    cc = nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [cc, *flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if r.stderr.strip():
            sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
