"""Build libgdr.so in-tree with nvcc for sm_103a (GB300) only, and _mixer.so, the Python binding of
the mixer's operators, with the host compiler against the installed PyTorch.

Each translation unit compiles in parallel; the shared library links the
static CUDA runtime so it loads on machines without a driver (the library's
symbols can be inspected there; kernels need a GB300).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgdr.so")
BINDING = os.path.join(PKG, "_mixer.so")
BINDING_SOURCE = "mixer_binding.cpp"

SOURCES = ["gdr_api.cu", "gdr_index.cu", "gdr_staged.cu", "gdr_fused.cu", "gdr_split.cu",
           "gdr_bwd.cu", "gdr_bwd_tc.cu", "gdr_mix_api.cu", "gdr_conv.cu", "gdr_ssm.cu",
           "gdr_ssm_wide.cu", "gdr_ssm_bwd.cu", "gdr_qk.cu", "gdr_delta_step.cu", "gdr_block_api.cu",
           "gdr_rec.cu", "gdr_rec_bwd.cu", "gdr_norm.cu", "gdr_attn.cu", "gdr_cache.cu"]
GENCODE = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
              "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps():
    """The compiled sources and every header they may include."""
    files = [os.path.join(CSRC, f) for f in SOURCES]
    files += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    files.append(os.path.join(INCLUDE, "gdr.h"))
    files.append(os.path.join(CSRC, BINDING_SOURCE))
    files.append(os.path.abspath(__file__))
    return files


def _stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return True
    # the older of the two: a build may have replaced the library and failed at the binding
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return any(os.path.getmtime(f) > t for f in _deps())


def _compile_binding() -> str:
    """The binding's object file; linked once libgdr.so is there."""
    import sysconfig

    import torch
    root = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(BUILD, os.path.splitext(BINDING_SOURCE)[0] + ".o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-I", root,
           "-I", os.path.join(root, "torch", "csrc", "api", "include"), "-I", cuda,
           "-c", os.path.join(CSRC, BINDING_SOURCE), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for {BINDING_SOURCE}:\n{r.stderr[-4000:]}")
    return obj


def _link_binding(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L", PKG, "-l:libgdr.so",
           "-Wl,-rpath,$ORIGIN", "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stderr[-4000:]}")
    os.replace(tmp, BINDING)


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    log = obj + ".log"
    cmd = [nvcc(), *GENCODE, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c",
           os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    with open(log, "w") as f:
        f.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr[-4000:]}")
    return obj


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every source, link libgdr.so and the binding; returns the library's path."""
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 4)) as ex:
        # the longest translation units first
        todo = sorted(SOURCES, key=lambda f: -os.path.getsize(os.path.join(CSRC, f)))
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(_compile, todo))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *GENCODE, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr[-4000:]}")
    os.replace(tmp, LIB)
    _link_binding(binding.result())
    if verbose:
        for src in SOURCES:
            log = os.path.join(BUILD, os.path.splitext(src)[0] + ".o.log")
            sys.stdout.write(open(log).read())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
