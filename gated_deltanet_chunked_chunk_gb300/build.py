"""Build libgdn.so for sm_103a with nvcc (no cmake, no torch extension machinery).

Every ``csrc/*.cu`` file is compiled to an object in parallel, then linked into
``_build/libgdn.so`` next to this file; ``csrc/gdn_torch.cpp``, the PyTorch
binding of the operators around the recurrence, becomes ``_build/_gdn_torch.so``,
linked to it.  Rebuilds only when a source or header is newer than the library,
or the binding was built for another PyTorch.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libgdn.so")
BINDING = os.path.join(BUILD, "_gdn_torch.so")
STAMP = os.path.join(BUILD, "_gdn_torch.for")  # the interpreter and PyTorch that BINDING was built for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: libgdn needs the CUDA toolkit to build")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.cpp")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)]


def _built_for() -> str:
    import torch
    return f"{sys.version} {torch.__version__} {torch.__file__}"


def binding_fits() -> bool:
    """Whether the binding was built for the running interpreter and PyTorch."""
    if not os.path.exists(STAMP):
        return False
    with open(STAMP) as f:
        return f.read() == _built_for()


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(BINDING) and binding_fits()):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return all(os.path.getmtime(p) <= t for p in _inputs())


def _binding_command(obj: str):
    """g++ command that compiles gdn_torch.cpp against the running interpreter's PyTorch."""
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    return [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-Wall",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
            "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"),
            "-c", os.path.join(CSRC, "gdn_torch.cpp"), "-o", obj]


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    srcs = sources()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(pair):
        src, obj = pair
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        return r.stderr

    binding_obj = os.path.join(BUILD, "gdn_torch.o")

    def compile_binding():
        r = subprocess.run(_binding_command(binding_obj), capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on gdn_torch.cpp:\n{r.stdout}\n{r.stderr}")
        return r.stderr

    with ThreadPoolExecutor(max_workers=min(16, len(srcs) + 1)) as ex:
        binding = ex.submit(compile_binding)
        for msg in ex.map(compile_one, zip(srcs, objs)):
            if verbose and msg:
                print(msg)
        msg = binding.result()
        if verbose and msg:
            print(msg)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-lcuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-shared", "-o", tmp, binding_obj, "-L", BUILD, "-lgdn", "-L", libs, "-ltorch_python",
           "-ltorch_cpu",
           "-ltorch_cuda", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    if os.path.exists(STAMP):  # from here on it is another binding's
        os.remove(STAMP)
    os.replace(tmp, BINDING)
    with open(tmp, "w") as f:
        f.write(_built_for())
    os.replace(tmp, STAMP)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
