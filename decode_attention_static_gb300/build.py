"""Build the CUDA library (libdecode_attn.so) for sm_103a with nvcc.

Each translation unit is compiled in parallel into _build/, then linked into
a shared library beside this file. cudart is linked statically, so the
library needs only the CUDA driver at run time.
"""
from __future__ import annotations

import concurrent.futures as cf
import contextlib
import hashlib
import os
import pathlib
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = pathlib.Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
INCLUDE = ROOT / "include"
BUILD_DIR = ROOT / "_build"
LIBRARY = PKG / "libdecode_attn.so"

SOURCES = ["abi.cu", "decode_f16.cu", "decode_bf16.cu", "decode_f16_rope.cu", "decode_bf16_rope.cu", "append.cu",
           "static_scratch.cu", "abi_paged.cu", "append_paged.cu", "cache_attn_f16.cu", "cache_attn_bf16.cu",
           "tree_attn.cu", "tree_attn_f16.cu", "tree_attn_bf16.cu", "abi_pages.cu", "page_pool.cu", "page_rows.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not pathlib.Path(exe).exists():
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")
    return exe


def _compile(src: pathlib.Path, obj: pathlib.Path, extra: list[str]) -> str:
    cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", str(src), "-o", str(obj)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src.name}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return r.stderr


def _stale(output: pathlib.Path) -> bool:
    if not output.exists():
        return True
    t = output.stat().st_mtime
    deps = list(CSRC.glob("*")) + list(INCLUDE.glob("*.h")) + [pathlib.Path(__file__)]
    return any(d.stat().st_mtime > t for d in deps)


def fastcall_path() -> pathlib.Path:
    """The fast path's module for this Python, torch and C header: it is bound to
    the first two, and its calls have the third one's argument lists."""
    import torch

    abi = hashlib.sha256((INCLUDE / "decode_attn.h").read_bytes()).hexdigest()[:8]
    return PKG / f"_fastcall.{sys.implementation.cache_tag}.torch-{torch.__version__}.{abi}.so"


def build_fastcall(force: bool = False) -> pathlib.Path | None:
    """Compile the binding's fast path if a source is newer than it; None (and
    a warning) where that does not work. No older module is left then: it calls
    the library by addresses, with the argument lists of its own sources."""
    import torch

    out = fastcall_path()
    if not force and not _stale(out):
        return out
    root = pathlib.Path(torch.__file__).parent
    tmp = out.with_name(out.name + f".tmp{os.getpid()}")
    try:
        cuda = pathlib.Path(nvcc()).parent.parent
        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{INCLUDE}",
               f"-I{root / 'include'}", f"-I{root / 'include/torch/csrc/api/include'}",
               f"-I{sysconfig.get_paths()['include']}", f"-I{cuda / 'include'}", str(CSRC / "fastcall.cpp"),
               "-o", str(tmp), f"-L{root / 'lib'}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python",
               f"-Wl,-rpath,{root / 'lib'}"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        why = f"\n{' '.join(cmd)}\n{r.stderr[-2000:]}" if r.returncode != 0 else None
    except (OSError, RuntimeError) as e:  # no compiler, no CUDA toolkit
        why = str(e)
    if why is not None:
        with contextlib.suppress(OSError):  # (a tree that cannot be written)
            out.unlink()
        warnings.warn(f"the binding's fast path was not built: {why}")
        return None
    os.replace(tmp, out)
    return out


def build_library(force: bool = False, verbose_ptxas: bool = False) -> pathlib.Path:
    """Compile and link the library (and the binding's fast path) if any source
    is newer than it."""
    with cf.ThreadPoolExecutor(max_workers=1) as fast:
        extra = fast.submit(build_fastcall, force)
        path = _build_library(force, verbose_ptxas)
        extra.result()
    return path


def _build_library(force: bool, verbose_ptxas: bool) -> pathlib.Path:
    if not force and not _stale(LIBRARY):
        return LIBRARY
    BUILD_DIR.mkdir(exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    objs = [BUILD_DIR / (s.replace(".cu", ".o")) for s in SOURCES]
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        logs = list(ex.map(lambda so: _compile(CSRC / so[0], so[1], extra), zip(SOURCES, objs)))
    if verbose_ptxas:
        for s, log in zip(SOURCES, logs):
            print(f"== {s}\n{log}")
    tmp = LIBRARY.with_name(LIBRARY.name + f".tmp{os.getpid()}")
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", str(tmp), *map(str, objs)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIBRARY)
    return LIBRARY


if __name__ == "__main__":
    print(build_library(force=True, verbose_ptxas="-v" in sys.argv))
