"""Build the native library ``lib/libgptq.so`` in-tree with nvcc for sm_100a, and the binding's native front
``lib/_binding.so`` (host code) with g++.

Usage: ``python -m post_weight_quantization_layer_b200.build`` (or ``build()``).
Cross-compiles on a machine without a GPU.
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libgptq.so")
BINDING = os.path.join(LIBDIR, "_binding.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING_ABI = os.path.join(LIBDIR, "_binding.abi")  # what the binding was built for
ROOT = os.path.dirname(PKG)

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "-prec-div=true", "-prec-sqrt=true",
    "-Xptxas", "-warn-spills",
]


def nvcc():
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def needs_build():
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h"))
    return any(os.path.getmtime(p) > t for p in deps)


def binding_abi():
    """What a build of the binding fits: the C++ side of one torch and one Python."""
    import torch

    return f"torch {torch.__version__} cxx11 {int(torch.compiled_with_cxx11_abi())} {sysconfig.get_config_var('SOABI')}"


def built_abi():
    """The same of the binding that is there; None where that is not known."""
    try:
        with open(BINDING_ABI) as f:
            return f.read().strip()
    except OSError:
        return None


def binding_needs_build():
    if not os.path.exists(BINDING) or built_abi() != binding_abi():
        return True
    t = os.path.getmtime(BINDING)
    return any(os.path.getmtime(p) > t for p in [BINDING_SRC] + glob.glob(os.path.join(ROOT, "include", "*.h")))


def binding_command(out):
    import torch

    base = os.path.dirname(torch.__file__)
    inc = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), sysconfig.get_paths()["include"]]
    abi = int(torch.compiled_with_cxx11_abi())
    return [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
            *(a for i in inc for a in ("-I", i)), BINDING_SRC, "-o", out, "-L", os.path.join(base, "lib"),
            "-Wl,-rpath," + os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    """Compile every CUDA source into one shared library, and the binding's front; returns the library's
    path.  Each is put in place as it succeeds: where the front cannot be built, the library is there all the same
    when this raises."""
    jobs = []
    if force or needs_build():
        jobs.append((LIB, lambda out: [nvcc(), *NVCC_FLAGS, *(extra_flags or []), "-I", os.path.join(ROOT, "include"),
                                       *sources(), "-o", out]))
    if force or binding_needs_build():
        jobs.append((BINDING, binding_command))
    if not jobs:
        return LIB
    os.makedirs(LIBDIR, exist_ok=True)
    running, failed = [], []
    for path, command in jobs:  # side by side
        try:
            cmd = command(path + ".tmp")
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            running.append((path, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)))
        except (OSError, ImportError, RuntimeError) as e:  # no compiler, no torch
            failed.append(f"{os.path.basename(path)}: {e}")
    for path, p in running:
        out, err = p.communicate()
        if p.returncode != 0:
            failed.append(f"{os.path.basename(path)}: compiler failed ({p.returncode}):\n{out}\n{err}")
            continue
        if verbose and (out or err):
            print(out + err, file=sys.stderr)
        os.replace(path + ".tmp", path)
        if path == BINDING:
            with open(BINDING_ABI, "w") as f:
                f.write(binding_abi() + "\n")
    if failed:
        raise RuntimeError("\n".join(failed))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
