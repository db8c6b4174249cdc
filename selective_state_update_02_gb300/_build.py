"""Builds libssu.so in-tree with nvcc for sm_103a (one -gencode; the translation units are
compiled in parallel, then linked into one shared library), and beside it the Python binding's
_marshal.so (host code alone)."""

from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
SOURCES = [CSRC / "ssu.cu", CSRC / "ssu_tokens.cu", CSRC / "ssu_copy.cu",
           CSRC / "ssu_prompt.cu", CSRC / "ssu_rotate.cu", CSRC / "ssu_attend.cu",
           CSRC / "ssu_host.cpp"]
HEADERS = [ROOT / "include" / "ssu.h", CSRC / "ssu_device.cuh", CSRC / "ssu_host.h",
           CSRC / "ssu_vec.cuh", CSRC / "ssu_stage.cuh",
           CSRC / "ssu_tokens.cuh", CSRC / "ssu_tokens_mma.cuh",
           CSRC / "ssu_prompt.cuh", CSRC / "ssu_prompt_mma.cuh",
           CSRC / "ssu_attend.cuh"]
OBJDIR = PKG / "_build"
LIB = PKG / "libssu.so"
MARSHAL_SOURCE = CSRC / "ssu_marshal.cpp"
MARSHAL = PKG / "_marshal.so"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and Path(cand).exists():
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libssu.so")


def compile_command(src: Path, obj: Path, extra: list[str] | None = None) -> list[str]:
    return [nvcc_path(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
            "-I", str(ROOT / "include"), "-I", str(CSRC), *(extra or []), "-c", str(src),
            "-o", str(obj)]


def link_command(objs: list[Path], out: Path) -> list[str]:
    return [nvcc_path(), *ARCH, "-shared", *[str(o) for o in objs], "-o", str(out)]


def marshal_command(out: Path) -> list[str]:
    import torch
    root = Path(torch.__file__).resolve().parent
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            "-I", str(ROOT / "include"), "-isystem", str(root / "include"),
            "-isystem", sysconfig.get_paths()["include"], str(MARSHAL_SOURCE), "-o", str(out),
            "-L", str(root / "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]


def _older(built: Path, sources: list[Path]) -> bool:
    return not built.exists() or any(p.stat().st_mtime > built.stat().st_mtime for p in sources)


def stale() -> bool:
    return _older(LIB, SOURCES + HEADERS) or _older(MARSHAL, [MARSHAL_SOURCE, HEADERS[0]])


def build(force: bool = False, extra: list[str] | None = None) -> Path:
    """Compile libssu.so and _marshal.so next to this file unless they are up to date."""
    if not (force or stale()):
        return LIB
    OBJDIR.mkdir(exist_ok=True)
    objs = [OBJDIR / (src.name + ".o") for src in SOURCES]
    procs = [subprocess.Popen(compile_command(src, obj, extra))
             for src, obj in zip(SOURCES, objs)]
    marshal = MARSHAL.with_name(f"_marshal.so.tmp{os.getpid()}")
    procs.append(subprocess.Popen(marshal_command(marshal)))
    codes = [p.wait() for p in procs]
    if any(codes):
        raise subprocess.CalledProcessError(max(codes), "nvcc, g++ (libssu sources)")
    os.replace(marshal, MARSHAL)
    tmp = LIB.with_name(f"libssu.so.tmp{os.getpid()}")
    subprocess.run(link_command(objs, tmp), check=True)
    os.replace(tmp, LIB)
    return LIB
