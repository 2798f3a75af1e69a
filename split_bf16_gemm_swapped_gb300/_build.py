"""Builds the package's native libraries in-tree (no pip install).

* ``_lib/libsplitk_sm103a.so``: the CUDA kernels and the C ABI declared in
  ``include/splitk.h``, compiled by nvcc for sm_103a only.
* ``_lib/libsynthetic.so``: the seeded input generator (plain C, gcc).
* ``_lib/_operators.so``: the Python binding of the operators around the
  projection (C++ on PyTorch's headers, g++), linked to the first.

Each is rebuilt when a source is newer than the library, and the binding also
when PyTorch or Python is another than it was built for.  Host code is
portable C/C++ (no x86 intrinsics, no -march=native), so the same sources
build on x86_64 and aarch64.
"""
from __future__ import annotations

import importlib.metadata
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
LIBDIR = PKG / "_lib"

SPLITK_LIB = LIBDIR / "libsplitk_sm103a.so"
SYNTHETIC_LIB = LIBDIR / "libsynthetic.so"
OPERATORS_LIB = LIBDIR / "_operators.so"
OPERATORS_STAMP = LIBDIR / "_operators.abi"         # what it was built for

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]

# Translation units of the CUDA library; compiled in parallel, linked once.
SPLITK_SOURCES = ["splitk_kernel.cu", "splitk_persistent.cu", "splitk_copy.cu", "splitk_host.cu",
                  "splitk_rows.cu", "splitk_i8.cu", "splitk_i8_stream.cu", "splitk_i8_tile.cu",
                  "splitk_logprobs.cu"]
SPLITK_HEADERS = ["splitk_device.cuh", "splitk_internal.h", "splitk_kernel_common.cuh", "splitk_i8.cuh"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not Path(cand).exists():
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build")
    return cand


def _stale(target: Path, deps) -> bool:
    if not target.exists():
        return True
    t = target.stat().st_mtime
    return any(Path(d).exists() and Path(d).stat().st_mtime > t for d in deps)


def _run(cmd, cwd=None):
    res = subprocess.run(cmd, cwd=cwd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(
            "build command failed:\n  " + " ".join(map(str, cmd)) + "\n" +
            res.stdout[-4000:] + res.stderr[-8000:])
    return res


def build_synthetic(force: bool = False) -> Path:
    LIBDIR.mkdir(parents=True, exist_ok=True)
    src = CSRC / "synthetic.c"
    if force or _stale(SYNTHETIC_LIB, [src]):
        tmp = SYNTHETIC_LIB.with_suffix(f".{os.getpid()}.tmp")
        _run(["gcc", "-O2", "-std=c11", "-Wall", "-Wextra", "-fPIC", "-shared",
              "-pthread", str(src), "-o", str(tmp), "-lm"])
        os.replace(tmp, SYNTHETIC_LIB)
    return SYNTHETIC_LIB


def build_splitk(force: bool = False, verbose_ptxas: bool = False) -> Path:
    LIBDIR.mkdir(parents=True, exist_ok=True)
    srcs = [CSRC / s for s in SPLITK_SOURCES]
    deps = srcs + [CSRC / h for h in SPLITK_HEADERS] + [INCLUDE / "splitk.h"]
    if not (force or _stale(SPLITK_LIB, deps)):
        return SPLITK_LIB
    nvcc = _nvcc()
    objdir = LIBDIR / f"obj.{os.getpid()}"
    objdir.mkdir(parents=True, exist_ok=True)
    common = [nvcc, *ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "-I", str(INCLUDE), "-I", str(CSRC)]
    if verbose_ptxas:
        common += ["-Xptxas", "-v"]

    def compile_one(src: Path):
        obj = objdir / (src.stem + ".o")
        res = _run(common + ["-c", str(src), "-o", str(obj)])
        return obj, res.stderr

    with ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        results = list(ex.map(compile_one, srcs))
    objs = [o for o, _ in results]
    tmp = SPLITK_LIB.with_suffix(f".{os.getpid()}.tmp")
    _run([nvcc, *ARCH_FLAGS, "-shared", "-o", str(tmp), *map(str, objs)])
    os.replace(tmp, SPLITK_LIB)
    shutil.rmtree(objdir, ignore_errors=True)
    if verbose_ptxas:
        for _, err in results:
            print(err)
    return SPLITK_LIB


def operators_abi() -> str:
    """The PyTorch (whose C++ types the binding uses) and the Python it is built
    for."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        from torch import __version__ as version
    return f"torch {version}, {sysconfig.get_config_var('SOABI')}"


def operators_built_for() -> str:
    return OPERATORS_STAMP.read_text() if OPERATORS_STAMP.exists() else ""


def build_operators(force: bool = False) -> Path:
    LIBDIR.mkdir(parents=True, exist_ok=True)
    src = CSRC / "operators_binding.cpp"
    abi = operators_abi()
    if not (force or _stale(OPERATORS_LIB, [src, INCLUDE / "splitk.h"]) or operators_built_for() != abi):
        return OPERATORS_LIB
    import torch
    home = Path(torch.__file__).resolve().parent
    cuda = Path(_nvcc()).resolve().parent.parent
    includes = [INCLUDE, sysconfig.get_paths()["include"], home / "include",
                home / "include" / "torch" / "csrc" / "api" / "include", cuda / "include"]
    tmp = OPERATORS_LIB.with_suffix(f".{os.getpid()}.tmp")
    _run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden", "-Wall",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          *[x for i in includes for x in ("-isystem" if str(i).startswith(str(home)) else "-I", str(i))],
          str(src), "-o", str(tmp), f"-L{LIBDIR}", f"-l:{SPLITK_LIB.name}", f"-L{home / 'lib'}",
          "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"])
    # (a build cut short between the two leaves no stamp: built again)
    OPERATORS_STAMP.unlink(missing_ok=True)
    os.replace(tmp, OPERATORS_LIB)
    OPERATORS_STAMP.write_text(abi)
    return OPERATORS_LIB


def build_all(force: bool = False) -> None:
    build_synthetic(force)
    build_splitk(force)
    build_operators(force)
