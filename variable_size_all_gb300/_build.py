"""Compile the CUDA library ``liba2av.so`` in-tree for sm_103a with nvcc."""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SOURCES = [os.path.join(PKG, "csrc", f) for f in ("a2av.cu", "dispatch.cu", "route.cu", "experts.cu",
                                                  "experts_mma.cu", "weighted.cu")]
HEADERS = [os.path.join(PKG, "csrc", f) for f in ("a2av_device.cuh", "a2av_handle.h",
                                                  "moe_device.cuh", "experts.cuh", "mma.cuh")]
INCLUDE = os.path.join(ROOT, "include")
LIBRARY = os.path.join(PKG, "liba2av.so")
MARSHAL_SOURCE = os.path.join(PKG, "csrc", "marshal.cpp")
MARSHAL = os.path.join(PKG, "_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))
MARSHAL_TORCH = os.path.join(PKG, "_marshal.torch")  # the torch it was compiled against
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the a2av library needs the CUDA toolkit to build")


def command(output: str = LIBRARY, extra=()) -> list:
    return [nvcc(), *ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
            "-shared", "-I", INCLUDE, *extra, "-o", output, *SOURCES]


def stale(output: str = LIBRARY) -> bool:
    if not os.path.exists(output):
        return True
    deps = SOURCES + HEADERS + [os.path.join(INCLUDE, f) for f in ("a2av.h", "a2av_moe.h")] + [__file__]
    return os.path.getmtime(output) < max(os.path.getmtime(d) for d in deps)


def _marshal_is_current(torch) -> bool:
    """Whether the compiled checks are of these sources and this torch, whose
    tensors they read as its headers lay them out."""
    try:
        with open(MARSHAL_TORCH) as f:
            made_for = f.read()
        return made_for == torch.__version__ and os.path.getmtime(MARSHAL) >= max(
            map(os.path.getmtime, (MARSHAL_SOURCE, os.path.join(INCLUDE, "a2av.h"),
                                   os.path.join(INCLUDE, "a2av_moe.h"))))
    except OSError:
        return False


def start_marshal(force: bool = False):
    """Begins to compile the binding's argument checks (csrc/marshal.cpp) against
    the installed torch; returns the process, or None when there is nothing to
    do.  Without torch, a compiler or the headers the binding does the checks itself."""
    try:
        import torch
    except ImportError:
        return None
    base = os.path.join(os.path.dirname(torch.__file__))
    include, python = os.path.join(base, "include"), sysconfig.get_paths()["include"]
    if not force and _marshal_is_current(torch):
        return None
    if shutil.which("g++") is None or not os.path.exists(os.path.join(python, "Python.h")):
        return None
    return subprocess.Popen(
        ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-w", "-I", INCLUDE, "-I", include, "-I",
         os.path.join(include, "torch", "csrc", "api", "include"), "-I", python,
         f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
         f'-DA2AV_TORCH="{torch.__version__}"', "-o", MARSHAL + ".tmp",
         MARSHAL_SOURCE, "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"])


def finish_marshal(process) -> None:
    """Puts the module in its place; where it did not compile, what was there is of
    other sources or another torch, and goes."""
    if process is None:
        return
    if process.wait() == 0:
        import torch
        os.replace(MARSHAL + ".tmp", MARSHAL)
        with open(MARSHAL_TORCH, "w") as f:
            f.write(torch.__version__)
    elif os.path.exists(MARSHAL):
        os.remove(MARSHAL)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """Build ``liba2av.so`` unless it is up to date; returns its path."""
    marshal = start_marshal(force)
    if force or stale():
        cmd = command(extra=extra)
        if verbose:
            print(" ".join(cmd))
        tmp = LIBRARY + ".tmp"
        subprocess.run(cmd[:-len(SOURCES) - 2] + ["-o", tmp, *SOURCES, "--threads", "0"],
                       check=True)
        os.replace(tmp, LIBRARY)
    finish_marshal(marshal)
    return LIBRARY


if __name__ == "__main__":
    build(force=True, verbose=True, extra=["-Xptxas", "-v"])
