"""Build libpagedkv.so (the CUDA library behind include/pagedkv.h) for sm_100a,
and ``_binding.so`` (the quick way from torch tensors to its host-bound calls).

``python -m paged_kv_cache_386_b200.build`` compiles in place with nvcc and g++;
the library links the CUDA runtime statically, so it loads without a GPU.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
LIB = PKG / "libpagedkv.so"
SOURCES = [CSRC / "pkv_api.cu", CSRC / "pkv_block_manager.cpp"]
HEADERS = sorted(CSRC.glob("*.cuh")) + [ROOT / "include" / "pagedkv.h"]
BINDING = PKG / "_binding.so"
BINDING_SOURCES = [CSRC / "pkv_binding.cpp", ROOT / "include" / "pagedkv.h"]

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def command(out: Path = LIB, verbose_ptxas: bool = False) -> list[str]:
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "-shared", "-Xcompiler", "-fPIC",
           "-cudart", "static", "-I", str(ROOT / "include"), "-I", str(CSRC),
           "-Xcompiler", "-Wall", "--expt-relaxed-constexpr"]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    return cmd + ["-o", str(out), *map(str, SOURCES)]


def binding_tag() -> str:
    """What an extension has to be built against to be used here."""
    import torch

    return f"torch {torch.__version__}, python {sys.version_info.major}.{sys.version_info.minor}"


def binding_command(out: Path = BINDING) -> list[str]:
    import torch

    torch_dir = Path(torch.__file__).resolve().parent
    cuda = Path(nvcc()).resolve().parent.parent
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            f'-DPKV_BUILT_FOR="{binding_tag()}"',
            "-I", str(ROOT / "include"), "-I", sysconfig.get_paths()["include"], "-I", str(torch_dir / "include"),
            "-I", str(cuda / "include"), "-o", str(out), str(BINDING_SOURCES[0]), "-L", str(torch_dir / "lib"),
            f"-Wl,-rpath,{torch_dir / 'lib'}", "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]


def stale(out: Path = LIB, sources=None) -> bool:
    if not out.exists():
        return True
    t = out.stat().st_mtime
    return any(p.stat().st_mtime > t for p in (SOURCES + HEADERS if sources is None else sources))


def build_binding(force: bool = False) -> bool:
    """The package runs without the extension (its calls then go through ctypes):
    where it cannot be built here, that is a warning, and none is left from another time."""
    if not force and not stale(BINDING, BINDING_SOURCES) and binding_tag().encode() in BINDING.read_bytes():
        return True
    try:
        subprocess.run(binding_command(BINDING), check=True)
        return True
    except (OSError, subprocess.CalledProcessError) as e:
        BINDING.unlink(missing_ok=True)
        warnings.warn(f"{BINDING.name} was not built, calls go through ctypes: {e}", stacklevel=2)
        return False


def build(force: bool = False, verbose_ptxas: bool = False) -> Path:
    if force or stale():
        subprocess.run(command(verbose_ptxas=verbose_ptxas), check=True)
    build_binding(force)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose_ptxas="-v" in sys.argv)
    print(LIB)
