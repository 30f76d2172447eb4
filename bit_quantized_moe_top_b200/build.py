"""Build the in-tree CUDA library ``libmoeq.so`` for sm_100a with nvcc, and, where
torch with CUDA is installed, the binding of the operators to torch tensors with the host
compiler. The library alone serves the C ABI."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libmoeq.so")
BINDING = os.path.join(HERE, "_binding.so")
BINDING_STAMP = os.path.join(HERE, "_binding.stamp")  # what the binding was built against
BUILD_DIR = os.path.join(ROOT, "_build")

SOURCES = ["moe_layer.cu", "route.cu", "relayout.cu", "decode_gemm.cu", "lowrank.cu", "noalloc.cu", "prefill_gemm.cu",
           "planner.cpp", "tileq.cu", "block_norm.cu", "grouped_tc.cu", "operators.cu"]
HEADERS = ["common.cuh", "decode_frag.cuh", "tc.cuh", "kernels.h", "ops.cuh", "grouped_loads.cuh", "grouped_form.h"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _inputs():
    srcs = [os.path.join(CSRC, s) for s in SOURCES]
    deps = srcs + [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(ROOT, "include", "moe_layer.h")]
    return srcs, deps


def _binding_inputs():
    return [os.path.join(CSRC, "binding.cpp"), os.path.join(ROOT, "include", "moe_layer.h")]


def _newer(out, deps) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(d) <= os.path.getmtime(out) for d in deps)


def _binding_key() -> str:
    """The torch and the Python whose headers and ABI the binding takes."""
    import sysconfig

    import torch
    return f"torch {torch.__version__} cxx11 {int(torch.compiled_with_cxx11_abi())} {sysconfig.get_config_var('SOABI')}"


def _have_torch() -> bool:
    try:
        import torch
    except ImportError:
        return False
    return torch.version.cuda is not None


def _binding_current() -> bool:
    if not _have_torch():
        return True  # nothing to bind to
    if not os.path.exists(BINDING_STAMP) or not _newer(BINDING, _binding_inputs()):
        return False
    with open(BINDING_STAMP) as f:
        return f.read() == _binding_key()


def up_to_date() -> bool:
    return _newer(LIB, _inputs()[1]) and _binding_current()


def build_binding() -> str:
    """The calls on torch tensors: host code against torch's headers, linked to libmoeq.so beside it."""
    import sysconfig

    import torch
    base = os.path.dirname(torch.__file__)
    tmp = BINDING + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-I", os.path.join(base, "include"), "-I", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"),
           "-I", os.path.join(ROOT, "include"), os.path.join(CSRC, "binding.cpp"), "-o", tmp,
           "-L", HERE, "-lmoeq", "-L", os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
           "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(BINDING_STAMP, "w") as f:
        f.write(_binding_key())
    return BINDING


def build(force: bool = False, verbose: bool = False, ptxas_v: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    if force or not _newer(LIB, _inputs()[1]):
        build_library(verbose, ptxas_v)
    if _have_torch() and (force or not _binding_current()):
        build_binding()
    return LIB


def build_library(verbose: bool = False, ptxas_v: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs, _ = _inputs()
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *FLAGS, "-c", src, "-o", obj]
        if ptxas_v:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_v:
            sys.stderr.write(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_v="-v" in sys.argv))
