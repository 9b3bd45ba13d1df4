"""Builds libgdn.so (the C-ABI library) in-tree with nvcc for sm_103a, and the torch binding of
the calls that are short enough for Python to matter (``_gdn_torch.so``, g++ against torch's
headers; it calls libgdn.so).

Each .cu file is compiled in parallel to an object, then linked into
``gated_delta_rule_07_gb300/_build/libgdn.so``.  Rebuilds only when a source or header is
newer than what was built of it, and the binding also when it was built for another torch or
Python.  Usage: ``python -m gated_delta_rule_07_gb300.build [--force]``.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libgdn.so")
TORCH_SRC = os.path.join(CSRC, "gdn_torch.cpp")
TORCH_LIB = os.path.join(BUILD, "_gdn_torch.so")
TORCH_FOR = TORCH_LIB + ".for"  # the torch and Python that it was built for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def cuda_lib_dir() -> str:
    base = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    for sub in ("lib64", "lib", "targets/sbsa-linux/lib", "targets/x86_64-linux/lib"):
        d = os.path.join(base, sub)
        if os.path.isdir(d):
            return d
    return os.path.join(base, "lib64")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newer(built: str, deps: list) -> bool:
    if not os.path.exists(built):
        return True
    t = os.path.getmtime(built)
    return any(os.path.getmtime(p) > t for p in deps)


def _library_stale() -> bool:
    return _newer(LIB, sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(
        os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def torch_build() -> str:
    """Which torch and Python a binding built now is for (torch itself is not imported)."""
    where = os.path.dirname(importlib.util.find_spec("torch").origin)
    with open(os.path.join(where, "version.py")) as f:
        return f"{sysconfig.get_config_var('EXT_SUFFIX')}\n{where}\n{f.read()}"


def _binding_stale() -> bool:
    if _newer(TORCH_LIB, [TORCH_SRC, os.path.join(INCLUDE, "gdn.h")]):
        return True
    if not os.path.exists(TORCH_FOR):
        return True
    with open(TORCH_FOR) as f:
        return f.read() != torch_build()


def torch_binding_command(out: str) -> list:
    """The g++ command that compiles gdn_torch.cpp (linked against libgdn.so beside it; torch's own
    libraries are in the process that imports it)."""
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    inc = [os.path.join(torch_dir, "include"),
           os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], INCLUDE]
    inc += [d for d in (os.path.join(cuda, "include"),
                        os.path.join(cuda, "targets", "sbsa-linux", "include"),
                        os.path.join(cuda, "targets", "x86_64-linux", "include"))
            if os.path.isdir(d)]
    lib = os.path.join(torch_dir, "lib")
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
            *[f"-I{d}" for d in inc], TORCH_SRC, "-o", out, f"-L{lib}", "-ltorch_python",
            "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{lib}"]


def build(force: bool = False, verbose: bool = False, extra: tuple = ()) -> str:
    library, binding_too = force or _library_stale(), force or _binding_stale()
    if not library and not binding_too:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    common = ["-O3", "-std=c++17", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC",
              f"-I{INCLUDE}", f"-I{CSRC}", "--expt-relaxed-constexpr", *extra]
    if verbose:
        common += ["-Xptxas", "-v"]
    procs, objs = [], []
    binding = TORCH_LIB + f".tmp{os.getpid()}"
    # (its references to libgdn.so are resolved when it is loaded, after that library)
    if binding_too:
        procs.append((TORCH_SRC, subprocess.Popen(torch_binding_command(binding),
                                                  stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                                  text=True)))
    for src in sources() if library else ():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        procs.append((src, subprocess.Popen([cc, *common, "-c", src, "-o", obj],
                                            stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                            text=True)))
    errors = []
    for src, p in procs:
        out, _ = p.communicate()
        if verbose or p.returncode:
            sys.stderr.write(out)
        if p.returncode:
            errors.append(src)
    if errors:
        raise RuntimeError(f"compiling failed for {errors}")
    if binding_too:
        os.replace(binding, TORCH_LIB)
        with open(TORCH_FOR, "w") as f:
            f.write(torch_build())
    if not library:
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    libdir = cuda_lib_dir()
    subprocess.run([cc, "-shared", *ARCH, "-cudart", "shared", "-o", tmp, *objs,
                    f"-L{libdir}", f"-Xlinker", f"-rpath={libdir}"], check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
