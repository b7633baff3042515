"""Builds libmoe_vq2.so in-tree with nvcc for sm_103a (one -gencode), one
translation unit per process, then links them, and the short way from Python to its
smallest calls (binding_path()) with g++ against PyTorch's headers.  The second is for
speed alone: where it cannot be built, a warning says so, and the calls go by ctypes."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe_vq2.so")
INCLUDE = os.path.join(ROOT, "include")
HEADER = os.path.join(INCLUDE, "moe_vq2.h")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe_vq2.so")
    return p


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _newest(files) -> float:
    return max(os.path.getmtime(f) for f in files)


def up_to_date() -> bool:
    """Whether libmoe_vq2.so is newer than its sources."""
    files = sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    return os.path.exists(LIB) and os.path.getmtime(LIB) >= _newest(files + [HEADER])


def binding_path() -> str:
    """The binding's file.  It is compiled against the headers of one Python and one
    PyTorch, which its name tells: another version's is another file."""
    import torch
    return os.path.join(PKG, f"moe_binding.{sysconfig.get_config_var('SOABI')}.torch-{torch.__version__}.so")


def binding_settled() -> bool:
    """Whether the binding, or the note that it could not be built here, is newer than
    its sources."""
    p = binding_path()
    newest = _newest([os.path.join(CSRC, "binding.cpp"), HEADER])
    return any(os.path.exists(f) and os.path.getmtime(f) >= newest for f in (p, p + ".failed"))


def build_binding() -> bool:
    """Builds the binding; where that fails, warns, leaves a note beside it (build()
    with force tries again) and returns False."""
    import torch
    p = binding_path()
    torch_dir = os.path.dirname(torch.__file__)
    try:
        cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
        cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", INCLUDE, "-I", os.path.join(cuda, "include"),
               "-I", sysconfig.get_paths()["include"], "-I", os.path.join(torch_dir, "include"),
               "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               os.path.join(CSRC, "binding.cpp"), "-o", p + ".tmp", "-L", os.path.join(torch_dir, "lib"),
               "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        fault = r.stderr if r.returncode != 0 else None
    except (OSError, RuntimeError) as e:  # (no g++, no toolkit)
        fault = str(e)
    if fault is None:
        os.replace(p + ".tmp", p)
        if os.path.exists(p + ".failed"):
            os.remove(p + ".failed")
        return True
    try:
        if os.path.exists(p):
            os.remove(p)  # (of older sources)
        with open(p + ".failed", "w") as f:
            f.write(fault)
    except OSError:  # (a folder that cannot be written)
        pass
    warnings.warn(f"{os.path.basename(p)} could not be built; its calls go by ctypes, which takes longer on the host "
                  f"(bit_vq_routed_gb300.build.build(force=True) tries again): {fault[:500]}", RuntimeWarning, stacklevel=2)
    return False


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and up_to_date():
        if not binding_settled():
            build_binding()
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        binding = ex.submit(build_binding) if force or not binding_settled() else None
        objs = list(ex.map(compile_one, sources()))
        if binding:
            binding.result()
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra=["-Xptxas", "-v"] if "-v" in sys.argv else []))
