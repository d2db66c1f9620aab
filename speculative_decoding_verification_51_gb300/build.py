"""Compile the CUDA library in-tree for sm_103a with nvcc.

Each translation unit under ``csrc/`` is compiled in parallel, then linked
into ``_build/libspecverify_<machine>.so`` (CUDA runtime linked statically).
``csrc/torch_ops.cpp`` becomes ``_build/specverify_torch_<machine>.so``, the
Python module that calls the library with torch tensors.  Both are rebuilt
when any source or header is newer than they are, the module also for
another torch.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import platform
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
SOURCES = ["plan.cu", "row_stats.cu", "sample.cu", "verify.cu", "tree.cu", "lmhead.cu", "host_io.cu",
           "rope.cu", "nodes.cu", "tree_attn.cu", "tree_attn_bf16.cu", "tree_attn_f16.cu",
           "tree_attn_e4m3.cu", "api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", f"-I{INCLUDE}"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.sep not in c or os.path.exists(c)):
            return c
    return "nvcc"


def lib_path() -> str:
    return os.path.join(BUILD, f"libspecverify_{platform.machine()}.so")


def ops_path() -> str:
    return os.path.join(BUILD, f"specverify_torch_{platform.machine()}.so")


def _inputs() -> list[str]:
    return (glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def extra_flags() -> list[str]:
    """Extra nvcc flags from SPEC_VERIFY_NVCC_EXTRA (e.g. launch-shape -D overrides)."""
    return os.environ.get("SPEC_VERIFY_NVCC_EXTRA", "").split()


def _stamp() -> str:
    return lib_path() + ".flags"


def _made_with() -> str:
    """What the library and the module depend on besides their sources."""
    import torch
    return " ".join([*extra_flags(), "torch", torch.__version__])


def up_to_date() -> bool:
    outs = [lib_path(), ops_path()]
    if not all(os.path.exists(p) for p in (*outs, _stamp())):
        return False
    if open(_stamp()).read() != _made_with():
        return False
    return min(os.path.getmtime(p) for p in outs) >= max(os.path.getmtime(p) for p in _inputs())


def _torch_flags() -> tuple[list[str], list[str]]:
    """(compiler, linker) flags of a module that calls torch."""
    import torch
    root = os.path.dirname(torch.__file__)
    inc = os.path.join(root, "include")
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    dirs = [sysconfig.get_paths()["include"], inc, os.path.join(inc, "torch", "csrc", "api", "include"),
            os.path.join(cuda, "include"), INCLUDE]
    libs = os.path.join(root, "lib")
    return ([f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"] + [f"-I{d}" for d in dirs],
            [f"-L{libs}", *(f"-l{n}" for n in ("torch_python", "torch", "torch_cuda", "torch_cpu", "c10_cuda", "c10")),
             f"-Wl,-rpath,{libs}"])


def build(force: bool = False, ptxas_verbose: bool = False) -> str:
    """Build the library if needed; return its path."""
    out = lib_path()
    if not force and up_to_date():
        return out
    objdir = os.path.join(BUILD, f"obj_{platform.machine()}")
    os.makedirs(objdir, exist_ok=True)
    extra = (["-Xptxas", "-v"] if ptxas_verbose else []) + extra_flags()

    def compile_one(src: str) -> tuple[str, str]:
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        return obj, r.stderr

    flags, libs = _torch_flags()
    ops_obj = os.path.join(objdir, "torch_ops.o")

    def compile_ops() -> None:
        r = subprocess.run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", *flags, "-c",
                            os.path.join(CSRC, "torch_ops.cpp"), "-o", ops_obj], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on torch_ops.cpp:\n{r.stderr}")

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        ops = ex.submit(compile_ops)
        results = list(ex.map(compile_one, SOURCES))
        ops.result()
    tmp = f"{out}.{os.getpid()}.tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, out)
    tmp = f"{ops_path()}.{os.getpid()}.tmp"
    r = subprocess.run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, ops_obj, f"-L{BUILD}",
                        f"-l:{os.path.basename(out)}", "-Wl,-rpath,$ORIGIN", *libs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, ops_path())
    with open(_stamp(), "w") as f:
        f.write(_made_with())
    if ptxas_verbose:
        for (_, log), src in zip(results, SOURCES):
            print(f"== {src}\n{log}")
    return out


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, ptxas_verbose="-v" in sys.argv))
