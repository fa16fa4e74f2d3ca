"""In-tree build of libspec.so (the C-ABI library) for sm_103a.

Each CUDA translation unit is compiled in parallel with nvcc and linked into
``libspec.so`` next to this file.  The CUDA runtime is linked statically, so
the library only needs the driver at run time.  Beside it, the binding's checks
of tensor arguments are compiled into the Python module ``_args``, which reads
torch's C++ objects: it is named for its Python and records the torch that it
was built with.  Rebuilds what a source or header is newer than, and ``_args``
for another torch.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
OBJDIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libspec.so")
ARGS = os.path.join(HERE, "_args" + sysconfig.get_config_var("EXT_SUFFIX"))
ARGS_FOR = os.path.join(OBJDIR, "args_for.txt")     # what ARGS was built for
SOURCES = ["spec_abi.cu", "spec_draft.cu", "spec_draft_slice.cu", "spec_verify.cu",
           "spec_verify_slice.cu", "spec_verify_redecide.cu", "spec_refine.cu", "spec_report.cu",
           "spec_sched.cu", "spec_tree.cu", "spec_tables.cu", "spec_cache.cu", "spec_attention.cu", "spec_attention_tc.cu",
           "spec_logprobs.cu"]
ARCH = "-gencode=arch=compute_103a,code=sm_103a"
NVCC_FLAGS = [ARCH, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
              "-I" + INCLUDE]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libspec")
    return cand


def _newer(than: str, *suffixes: str) -> bool:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(suffixes)]
    if ".cu" in suffixes:
        files.append(os.path.join(INCLUDE, "spec.h"))
    t = os.path.getmtime(than)
    return any(os.path.getmtime(f) > t for f in files)


def built_for() -> str:
    """The torch whose objects ``_args`` reads."""
    import torch
    return f"torch {torch.__version__} {torch.version.git_version}"


def _lib_stale() -> bool:
    return not os.path.exists(LIB) or _newer(LIB, ".cu", ".cuh")


def _args_stale() -> bool:
    if not (os.path.exists(ARGS) and os.path.exists(ARGS_FOR)) or _newer(ARGS, ".cpp"):
        return True
    with open(ARGS_FOR) as f:
        return f.read() != built_for()


def is_stale() -> bool:
    return _lib_stale() or _args_stale()


def _build_args() -> None:
    import torch
    home = os.path.dirname(torch.__file__)
    inc = os.path.join(home, "include")
    tmp = ARGS + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           f'-DSPEC_BUILT_FOR="{built_for()}"',
           "-I" + sysconfig.get_paths()["include"], "-I" + inc,
           "-I" + os.path.join(inc, "torch", "csrc", "api", "include"),
           os.path.join(CSRC, "spec_args.cpp"), "-o", tmp, "-L" + os.path.join(home, "lib"),
           "-lc10", "-ltorch_cpu", "-ltorch_python"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on spec_args.cpp:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, ARGS)
    with open(ARGS_FOR, "w") as f:
        f.write(built_for())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libspec.so and _args; returns the library's path."""
    os.makedirs(OBJDIR, exist_ok=True)
    args_stale = force or _args_stale()
    if not force and not _lib_stale():
        if args_stale:
            _build_args()
        return LIB
    nvcc = _nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(OBJDIR, src.replace(".cu", ".o"))
        cmd = [nvcc, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
        if verbose:
            print(res.stdout + res.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        args = ex.submit(_build_args) if args_stale else None
        objs = list(ex.map(compile_one, SOURCES))
        if args:
            args.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc, ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
