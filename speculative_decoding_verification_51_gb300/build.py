"""Compile the CUDA library in-tree for sm_103a with nvcc.

Each translation unit under ``csrc/`` is compiled in parallel, then linked
into ``_build/libspecverify_<machine>.so`` (CUDA runtime linked statically).
``csrc/torch_ops.cpp`` becomes ``_build/specverify_torch_<machine>.so``, the
Python module that calls the library with torch tensors; without torch there
is the library alone.  Either is rebuilt when one of its sources or headers is
newer than it is, the module also for another torch.
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
           "tree_attn_e4m3.cu", "norm.cu", "norm_e4m3.cu", "prompt.cu", "prompt_attn_bf16.cu", "prompt_attn_f16.cu", "logprob.cu",
           "api.cu"]
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


def _inputs(*endings: str) -> list[str]:
    return [p for e in endings for p in glob.glob(os.path.join(CSRC, "*." + e))] + glob.glob(os.path.join(INCLUDE, "*.h"))


def extra_flags() -> list[str]:
    """Extra nvcc flags from SPEC_VERIFY_NVCC_EXTRA (e.g. launch-shape -D overrides)."""
    return os.environ.get("SPEC_VERIFY_NVCC_EXTRA", "").split()


def _torch_version() -> str | None:
    """None without torch: then there is the library alone."""
    try:
        import torch
    except ImportError:
        return None
    return torch.__version__


def _fresh(out: str, made_with: str, inputs: list[str]) -> bool:
    """Whether `out` is there, made with the same as now and newer than its inputs."""
    stamp = out + ".flags"
    if not os.path.exists(out) or not os.path.exists(stamp) or open(stamp).read() != made_with:
        return False
    return os.path.getmtime(out) >= max(os.path.getmtime(p) for p in inputs)


def _put(tmp: str, out: str, made_with: str) -> None:
    os.replace(tmp, out)
    with open(out + ".flags", "w") as f:
        f.write(made_with)


def _stale() -> tuple[bool, bool]:
    """Whether the library, and the module, have to be made."""
    torch_version = _torch_version()
    return (not _fresh(lib_path(), " ".join(extra_flags()), _inputs("cu", "cuh")),
            torch_version is not None and not _fresh(ops_path(), torch_version, _inputs("cpp")))


def up_to_date() -> bool:
    return not any(_stale())


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
    """Build what is needed of the library and the module; return the library's path."""
    out, module = lib_path(), ops_path()
    make_lib, make_module = _stale()
    if force:
        make_lib, make_module = True, _torch_version() is not None
    if not make_lib and not make_module:
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

    cxx, ops_obj = os.environ.get("CXX", "g++"), os.path.join(objdir, "torch_ops.o")

    def compile_ops() -> list[str]:
        flags, libs = _torch_flags()
        r = subprocess.run([cxx, "-O2", "-std=c++17", "-fPIC", *flags, "-c", os.path.join(CSRC, "torch_ops.cpp"),
                            "-o", ops_obj], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on torch_ops.cpp:\n{r.stderr}")
        return libs

    def link(cmd: list[str], to: str, made_with: str) -> None:
        tmp = f"{to}.{os.getpid()}.tmp"
        r = subprocess.run([*cmd, "-shared", "-o", tmp], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
        _put(tmp, to, made_with)

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        ops = ex.submit(compile_ops) if make_module else None
        results = list(ex.map(compile_one, SOURCES)) if make_lib else []
        if make_lib:  # whatever becomes of the module
            link([nvcc(), *ARCH, *[o for o, _ in results]], out, " ".join(extra_flags()))
        if make_module:
            libs = ops.result()
            link([cxx, ops_obj, f"-L{BUILD}", f"-l:{os.path.basename(out)}", "-Wl,-rpath,$ORIGIN", *libs], module,
                 _torch_version())
    if ptxas_verbose:
        for (_, log), src in zip(results, SOURCES):
            print(f"== {src}\n{log}")
    return out


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, ptxas_verbose="-v" in sys.argv))
