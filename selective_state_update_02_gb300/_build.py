"""Builds libssu.so in-tree with nvcc for sm_103a (one -gencode; the translation units are
compiled in parallel, then linked into one shared library), and beside it the Python binding's
_marshal.so (host code alone)."""

from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
import warnings
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
SOURCES = [CSRC / "ssu.cu", CSRC / "ssu_tokens.cu", CSRC / "ssu_copy.cu",
           CSRC / "ssu_prompt.cu", CSRC / "ssu_rotate.cu", CSRC / "ssu_attend.cu",
           CSRC / "ssu_delta.cu", CSRC / "ssu_norm.cu", CSRC / "ssu_host.cpp"]
HEADERS = [ROOT / "include" / "ssu.h", CSRC / "ssu_device.cuh", CSRC / "ssu_host.h",
           CSRC / "ssu_vec.cuh", CSRC / "ssu_stage.cuh",
           CSRC / "ssu_tokens.cuh", CSRC / "ssu_tokens_mma.cuh",
           CSRC / "ssu_prompt.cuh", CSRC / "ssu_prompt_mma.cuh",
           CSRC / "ssu_attend.cuh", CSRC / "ssu_delta.cuh", CSRC / "ssu_delta_mma.cuh",
           CSRC / "ssu_tc.cuh", CSRC / "ssu_tma.h"]
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


def _library_stale() -> bool:
    return _older(LIB, SOURCES + HEADERS)


def _marshal_note() -> Path:
    return MARSHAL.with_name("_marshal.built_for")


def marshal_wants() -> str:
    """What _marshal.so must have been built for: it uses torch's C++ classes and Python's ABI, so
    that one of another version may crash instead of failing."""
    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def marshal_built_for() -> str:
    """What _marshal.so was built for; "" if that is not known."""
    try:
        return _marshal_note().read_text()
    except OSError:
        return ""


def _marshal_stale() -> bool:
    try:
        wanted = marshal_wants()
    except ImportError:
        return True
    return _older(MARSHAL, [MARSHAL_SOURCE, HEADERS[0]]) or marshal_built_for() != wanted


def stale() -> bool:
    return _library_stale() or _marshal_stale()


def _build_library(extra: list[str] | None) -> None:
    OBJDIR.mkdir(exist_ok=True)
    objs = [OBJDIR / (src.name + ".o") for src in SOURCES]
    procs = [subprocess.Popen(compile_command(src, obj, extra))
             for src, obj in zip(SOURCES, objs)]
    codes = [p.wait() for p in procs]
    if any(codes):
        raise subprocess.CalledProcessError(max(codes), "nvcc (libssu sources)")
    tmp = LIB.with_name(f"libssu.so.tmp{os.getpid()}")
    subprocess.run(link_command(objs, tmp), check=True)
    os.replace(tmp, LIB)


def _start_marshal(out: Path) -> subprocess.Popen | None:
    try:
        return subprocess.Popen(marshal_command(out))
    except (ImportError, OSError):  # no torch, no g++
        return None


def build(force: bool = False, extra: list[str] | None = None) -> Path:
    """Compile libssu.so and _marshal.so next to this file unless they are up to date.  nvcc alone is
    enough for libssu.so, which the C ABI and every call but the prompt, rotation, attention,
    delta-rule and norm calls of the Python binding are content with: where _marshal.so cannot be built (it needs
    g++ and the headers of Python and torch), that is a warning."""
    library, binding = force or _library_stale(), force or _marshal_stale()
    tmp = MARSHAL.with_name(f"_marshal.so.tmp{os.getpid()}")
    marshal = _start_marshal(tmp) if binding else None
    try:
        if library:
            _build_library(extra)
    finally:
        built = marshal is not None and marshal.wait() == 0
        if built:
            _marshal_note().unlink(missing_ok=True)
            os.replace(tmp, MARSHAL)
            _marshal_note().write_text(marshal_wants())
        elif binding:
            tmp.unlink(missing_ok=True)
            MARSHAL.unlink(missing_ok=True)  # what is there is of other sources
    if binding and not built:
        warnings.warn("_marshal.so could not be built: the prompt, rotation, attention, delta-rule "
                      "and norm calls are not available from Python", stacklevel=2)
    return LIB
