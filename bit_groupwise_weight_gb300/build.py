"""Build liblowbit.so in-tree with nvcc for sm_103a (GB300), and beside it the
extension module _lowbit_torch (csrc/binding.cpp: the hot path of the decoder
operators' Python binding, against the installed PyTorch's headers).

Each .cu under csrc/ compiles to an object in parallel; the objects link into
one shared library with the CUDA runtime linked statically, so the library
loads on a machine without a GPU (only the first CUDA call needs the driver).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
BUILD = PKG / "_build"
LIB = BUILD / "liblowbit.so"

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++20", "-lineinfo", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", "-Wno-deprecated-gpu-targets"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and Path(cand).exists():
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build liblowbit")


def sources() -> list[Path]:
    return sorted(CSRC.glob("*.cu"))


def _deps() -> list[Path]:
    return (sources() + sorted(CSRC.glob("*.cuh")) + sorted(CSRC.glob("*.cpp")) + sorted(INCLUDE.glob("*.h"))
            + [Path(__file__)])


def binding() -> Path:
    """The extension module's file, named after the PyTorch and the Python that it is compiled
    against, so that another one's is neither loaded nor taken for up to date."""
    import torch
    commit = (torch.version.git_version or "")[:8]
    return BUILD / f"_lowbit_torch-{torch.__version__}-{commit}{sysconfig.get_config_var('EXT_SUFFIX')}"


def up_to_date() -> bool:
    module = binding()
    if not LIB.exists() or not module.exists():
        return False
    t = min(LIB.stat().st_mtime, module.stat().st_mtime)
    return all(p.stat().st_mtime <= t for p in _deps())


def build_binding(verbose: bool = False) -> None:
    """The extension module: host code only, linked to PyTorch and not to liblowbit."""
    import torch
    root = Path(torch.__file__).resolve().parent
    cuda = Path(nvcc()).resolve().parent.parent
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        raise RuntimeError("a C++ compiler is needed to build _lowbit_torch")
    module = binding()
    tmp = module.with_suffix(f".{os.getpid()}.tmp")
    cmd = [cxx, "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{p}" for p in (INCLUDE, root / "include", root / "include/torch/csrc/api/include",
                                sysconfig.get_paths()["include"], cuda / "include")),
           str(CSRC / "binding.cpp"), "-o", str(tmp), f"-L{root / 'lib'}", "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python", f"-Wl,-rpath,{root / 'lib'}"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the C++ compiler failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, module)


def build(force: bool = False, verbose: bool = False, extra_flags: tuple[str, ...] = ()) -> Path:
    if not force and not extra_flags and up_to_date():
        return LIB
    BUILD.mkdir(parents=True, exist_ok=True)
    cc = nvcc()

    def compile_one(src: Path) -> Path:
        obj = BUILD / (src.stem + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra_flags, "-I", str(INCLUDE), "-c", str(src), "-o", str(obj)]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src.name}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with ThreadPoolExecutor(max_workers=max(1, min(len(sources()) + 1, os.cpu_count() or 4))) as ex:
        module = ex.submit(build_binding, verbose)
        objs = list(ex.map(compile_one, sources()))
        module.result()
    tmp = LIB.with_suffix(f".{os.getpid()}.tmp")
    cmd = [cc, *ARCH, "-shared", "-cudart", "static", *map(str, objs), "-o", str(tmp)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
