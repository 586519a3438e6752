"""Builds libgdr.so in-tree with nvcc for sm_103a (GB300).

Each translation unit under csrc/ is compiled in parallel into _build/, then
linked into _build/libgdr.so (CUDA runtime linked statically, so loading the
library needs no libcudart on the path and no GPU).  A unit is rebuilt only
when it or a header under csrc/ or include/ is newer than its object file.

binding/layer_binding.cpp, the torch binding of the layer operators, is a host
file: it becomes _build/_gdr_layer.so with the host compiler against the
installed torch's headers, beside the units of libgdr, which it links to.
_gdr_layer.so.for says which torch and Python it was built for; for another one
it is built again.
libgdr itself needs no torch: run as a script, this file builds it without.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libgdr.so")
BINDING_SRC = os.path.join(PKG, "binding", "layer_binding.cpp")
BINDING = os.path.join(BUILD, "_gdr_layer.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: libgdr needs the CUDA toolkit to build")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _headers_mtime() -> float:
    hs = glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(h) for h in hs), default=0.0)


def _binding_target():
    """The torch and Python that a binding is for: where torch lies, its version file and Python's ABI, all without importing
    torch; None without a torch."""
    torch = importlib.util.find_spec("torch")
    if torch is None:
        return None
    home = os.path.dirname(torch.origin)
    with open(os.path.join(home, "version.py")) as f:
        return "\n".join([sysconfig.get_config_var("SOABI") or sys.version, home, f.read()])


def _binding_is_for(target: str) -> bool:
    """Whether the built binding is newer than its sources and was built for this torch and Python."""
    if not os.path.exists(BINDING) or not os.path.exists(BINDING + ".for"):
        return False
    if os.path.getmtime(BINDING) < max(os.path.getmtime(BINDING_SRC), os.path.getmtime(os.path.join(INCLUDE, "gdr.h"))):
        return False
    with open(BINDING + ".for") as f:
        return f.read() == target


def _binding_commands(obj: str, out: str):
    """The compile and link commands of the layer binding, for the torch and Python that run this."""
    import torch
    home = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    cxx = shutil.which("g++") or "g++"
    return ([cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={abi}", "-I", INCLUDE,
             "-I", os.path.join(home, "include"), "-I", os.path.join(home, "include", "torch", "csrc", "api", "include"),
             "-I", sysconfig.get_paths()["include"], "-I", cuda, "-c", BINDING_SRC, "-o", obj],
            [cxx, "-shared", "-o", out, obj, "-L", BUILD, "-lgdr", "-L", os.path.join(home, "lib"), "-lc10", "-lc10_cuda",
             "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + os.path.join(home, "lib")])


def build(verbose: bool = False, force: bool = False, extra_flags=None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    hdr = _headers_mtime()
    flags = NVCC_FLAGS + list(extra_flags or [])
    jobs = []
    objs = []
    for src in _sources():
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        objs.append(obj)
        if force or not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(src), hdr):
            jobs.append([nvcc, *ARCH, *flags, "-c", src, "-o", obj])

    built_for = _binding_target()
    # without torch there is nothing to bind to, and libgdr is built alone
    new_binding = built_for is not None and (force or not _binding_is_for(built_for))
    units = len(jobs)
    if new_binding:
        binding_obj = os.path.join(BUILD, "layer_binding.o")
        compile_binding, link_binding = _binding_commands(binding_obj, BINDING + f".tmp{os.getpid()}")
        jobs.append(compile_binding)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"the compiler failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)

    if jobs:
        with ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            list(ex.map(run, jobs))
    if units or not os.path.exists(LIB) or force:
        tmp = LIB + f".tmp{os.getpid()}"
        run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    if new_binding:
        run(link_binding)
        with open(BINDING + ".for", "w"):                # says nothing of the new file until that lies in its place
            pass
        os.replace(BINDING + f".tmp{os.getpid()}", BINDING)
        with open(BINDING + ".for", "w") as f:
            f.write(built_for)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, force="--force" in sys.argv))
