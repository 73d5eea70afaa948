"""Build libmol.so (the MoL LoRA CUDA library) in-tree with nvcc for sm_103a.

Beside it _block_native.so, the native calls of the MoE block's binding: plain C++ against
PyTorch's headers. Without it (no compiler for them, or built for another PyTorch or Python) the
binding takes its Python path, which gives the same results."""

from __future__ import annotations

import os
import platform
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG_DIR, "libmol.so")
# The same sources with device-side index checks (MOL_CHECKED): a diagnostic build.
CHECKED_LIB_PATH = os.path.join(PKG_DIR, "libmol_checked.so")
NATIVE_PATH = os.path.join(PKG_DIR, "_block_native.so")
NATIVE_STAMP = NATIVE_PATH + ".stamp"  # what it was built for
NATIVE_SOURCE = os.path.join(CSRC, "mol_block_py.cpp")

SOURCES = ["mol_abi.cu", "mol_align.cu", "mol_lora.cu", "mol_umma.cu", "mol_stage.cu",
           "mol_expand_tc.cu", "mol_block_abi.cu", "mol_block.cu", "mol_moe.cu",
           "mol_moe_bf16.cu", "mol_moe_w4_32.cu", "mol_moe_w4_64.cu", "mol_moe_w4_128.cu",
           "mol_attn_abi.cu", "mol_rope.cu", "mol_attend.cu", "mol_attend_tc.cu",
           "mol_attend_wide.cu"]
HEADERS = ["mol_device.cuh", "mol_internal.h", "mol_tc.cuh", "mol_moe.h", "mol_moe.cuh",
           "mol_attend.h", "mol_attend.cuh"]
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the MoL library needs the CUDA toolkit to build")


def _built_for() -> str:
    """What the native calls' binary interface depends on."""
    import torch

    return f"python {sys.version}\ntorch {torch.__version__}\n{platform.machine()}\n"


def native_current() -> bool:
    """Whether the native calls were built for this Python, PyTorch and machine."""
    try:
        with open(NATIVE_STAMP) as f:
            return f.read() == _built_for()
    except OSError:
        return False


def _stale(path: str) -> bool:
    if not os.path.exists(path) or (path == NATIVE_PATH and not native_current()):
        return True
    t = os.path.getmtime(path)
    sources = ([NATIVE_SOURCE] if path == NATIVE_PATH
               else [os.path.join(CSRC, f) for f in SOURCES + HEADERS])
    deps = sources + [
        os.path.join(INCLUDE, "mol.h"), os.path.join(INCLUDE, "mol_block.h"),
        os.path.join(INCLUDE, "mol_attn.h"), os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps)


def _command(out: str, checked: bool, verbose: bool) -> list:
    cmd = [nvcc_path(), "-O3", "-std=c++17", *ARCH_FLAGS, "-lineinfo", "-Xcompiler", "-fPIC",
           "-shared", "-I", INCLUDE, "--threads", "4", "-o", out]
    if checked:
        cmd += ["-DMOL_CHECKED"]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    return cmd + [os.path.join(CSRC, f) for f in SOURCES]


def _native_command(out: str) -> list:
    import torch

    home = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include")
    dirs = [INCLUDE, os.path.join(home, "include"),
            os.path.join(home, "include", "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], cuda]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[a for d in dirs for a in ("-I", d)], NATIVE_SOURCE, "-o", out,
            "-L", os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def build_library(force: bool = False, verbose: bool = False, checked: bool = False) -> str:
    """Compile the translation units (nvcc --threads 4) into one shared library.

    checked=True builds libmol_checked.so, the same kernels with the device-side
    index checks compiled in."""
    path = CHECKED_LIB_PATH if checked else LIB_PATH
    if not force and not _stale(path):
        return path
    tmp = path + f".tmp{os.getpid()}"
    res = subprocess.run(_command(tmp, checked, verbose), capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    if verbose:
        print(res.stdout + res.stderr)
    os.replace(tmp, path)
    return path


def build_all(force: bool = False) -> tuple:
    """Build the release and the checked library and the native calls at the same time."""
    jobs = []

    def start(path, tmp, cmd):
        jobs.append((path, tmp, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                                 stderr=subprocess.STDOUT, text=True)))

    for checked in (False, True):
        path = CHECKED_LIB_PATH if checked else LIB_PATH
        if force or _stale(path):
            tmp = path + f".tmp{os.getpid()}"
            start(path, tmp, _command(tmp, checked, False))
    native = os.path.basename(NATIVE_PATH)
    try:
        if force or _stale(NATIVE_PATH):
            tmp = NATIVE_PATH + f".tmp{os.getpid()}"
            start(NATIVE_PATH, tmp, _native_command(tmp))
    except (OSError, ImportError, AttributeError) as e:  # no g++, or no PyTorch to build against
        warnings.warn(f"{native} was not built: {e!r}")
    errors = []
    for path, tmp, proc in jobs:
        out, _ = proc.communicate()
        if proc.returncode != 0 and path == NATIVE_PATH:
            warnings.warn(f"{native} was not built:\n{out}")
        elif proc.returncode != 0:
            errors.append(f"{os.path.basename(path)}:\n{out}")
        elif path == NATIVE_PATH:
            with open(NATIVE_STAMP, "w") as f:  # (empty while the file is another's)
                f.flush()
                os.replace(tmp, path)
                f.write(_built_for())
        else:
            os.replace(tmp, path)
    if errors:
        raise RuntimeError("nvcc failed:\n" + "\n".join(errors))
    return LIB_PATH, CHECKED_LIB_PATH


if __name__ == "__main__":
    print(build_library(force=True, verbose=True))
