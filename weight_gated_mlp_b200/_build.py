"""Build of the CUDA library ``libittt.so`` (sm_100a) and of the argument
marshalling module ``_marshal.so`` next to this file.

``python -m weight_gated_mlp_b200._build`` compiles ``csrc/api.cu`` (which
includes every kernel header) with nvcc into a shared library exporting the
C ABI of ``include/ittt.h``.  The CUDA runtime is linked statically.
``csrc/marshal.cpp`` (g++, torch's and Python's headers) becomes the Python module
through which the operators around the layer are called; where these are
missing, the library is built all the same and the module is left out.
"""

from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libittt.so")
SOURCES = [os.path.join(PKG, "csrc", "api.cu")]
DEPS = [os.path.join(PKG, "csrc", n) for n in sorted(os.listdir(os.path.join(PKG, "csrc")))
        if not n.endswith(".cpp")] + [os.path.join(ROOT, "include", "ittt.h")]
MARSHAL = os.path.join(PKG, "_marshal.so")
MARSHAL_SOURCE = os.path.join(PKG, "csrc", "marshal.cpp")


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def command(out: str = LIB, verbose_ptxas: bool = False) -> list:
    cmd = [nvcc_path(), "-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a",
           "-lineinfo", "-Xcompiler", "-fPIC", "-shared", "-I", os.path.join(ROOT, "include"),
           "-o", out] + SOURCES
    if verbose_ptxas:
        cmd.insert(1, "-Xptxas=-v")
    return cmd


def marshal_command(out: str = MARSHAL) -> list:
    import torch

    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    lib = os.path.join(base, "lib")
    return [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(base, "include"),
            "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(cuda, "include"), "-I", sysconfig.get_paths()["include"],
            "-o", out, MARSHAL_SOURCE, "-L", lib, "-ltorch_python", "-ltorch", "-ltorch_cpu",
            "-ltorch_cuda", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{lib}"]


def marshal_lacks() -> Optional[str]:
    """What the marshalling module needs and is not here; None: nothing."""
    if importlib.util.find_spec("torch") is None:
        return "torch"
    if shutil.which("g++") is None:
        return "g++"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python's headers"
    return None


def marshal_key() -> str:
    """What the module is built against: Python's and torch's versions.  It stands in
    a file beside the module, which is made again where they change."""
    try:
        torch_version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        from torch import __version__ as torch_version
    return f"{sysconfig.get_config_var('SOABI')}, torch {torch_version}"


def marshal_up_to_date() -> bool:
    try:
        with open(MARSHAL + ".key") as f:
            built = f.read()
    except OSError:
        return False
    return built == marshal_key() and newer(MARSHAL, [MARSHAL_SOURCE, os.path.join(ROOT, "include", "ittt.h")])


def newer(target: str, sources) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(p) <= t for p in sources if os.path.exists(p))


def up_to_date() -> bool:
    return newer(LIB, DEPS)


def run(cmd: list, target: str, what: str):
    """Run a compiler command that writes target + ".tmp", then move it into place."""
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"{what} failed:\n" + res.stdout + res.stderr)
    os.replace(target + ".tmp", target)
    return res


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if force or not up_to_date():
        res = run(command(LIB + ".tmp", verbose_ptxas), LIB, "nvcc")
        if verbose_ptxas:
            sys.stderr.write(res.stderr)
    lacks = marshal_lacks()
    if lacks:
        sys.stderr.write(f"{MARSHAL} not built, and with it linear, causal_conv and selective_scan in "
                         f"Python: no {lacks}\n")
    elif force or not marshal_up_to_date():
        run(marshal_command(MARSHAL + ".tmp"), MARSHAL, "g++")
        with open(MARSHAL + ".key", "w") as f:
            f.write(marshal_key())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
