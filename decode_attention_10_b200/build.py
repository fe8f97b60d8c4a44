"""Build libmfa.so (the C-ABI library) in-tree with nvcc for sm_100a, and mfa_torch.so (the
binding of its chunk calls for torch tensors) with the host compiler.

    python -m decode_attention_10_b200.build [--verbose]

Both are written next to this file so that they travel with the source tree.
"""

import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmfa.so")
BINDING = os.path.join(HERE, "mfa_torch.so")
BINDING_FOR = os.path.join(ROOT, "_build", "mfa_torch.txt")
SOURCES = ["abi.cu", "query_path.cu", "gemm_tc.cu", "attention_tc.cu", "out_proj.cu", "noalloc.cu",
           "selftest.cu", "split_plan.cu", "rope_append.cu", "chunk_attn.cu"]
HEADERS = ["mfa_internal.cuh", "attn_plan.cuh", "sm100.cuh", "chunk.cuh"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def nvcc_flags():
    return ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
            "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
            "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    deps.append(os.path.join(ROOT, "include", "mfa.h"))
    deps.append(os.path.abspath(__file__))
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def _built_for() -> str:
    """What the binding was last built for (see build_binding)."""
    try:
        with open(BINDING_FOR) as f:
            return f.read()
    except OSError:
        return ""


def build_binding(force: bool = False, verbose: bool = False) -> str:
    import torch
    src = os.path.join(CSRC, "binding.cpp")
    deps = [src, os.path.join(ROOT, "include", "mfa.h"), os.path.abspath(__file__)]
    # it fits one torch and one Python only
    built_for = f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}\n"
    if (not force and os.path.exists(BINDING) and _built_for() == built_for
            and all(os.path.getmtime(d) <= os.path.getmtime(BINDING) for d in deps)):
        return BINDING
    base = os.path.dirname(torch.__file__)
    inc = [os.path.join(base, "include"),
           os.path.join(base, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include"),
           sysconfig.get_paths()["include"]]
    libs = os.path.join(base, "lib")
    tmp = f"{BINDING}.{os.getpid()}.tmp"  # (two ranks may build at once)
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-I{i}" for i in inc], src, "-o", tmp, "-L", libs, "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, BINDING)
    os.makedirs(os.path.dirname(BINDING_FOR), exist_ok=True)
    tmp = f"{BINDING_FOR}.{os.getpid()}.tmp"
    with open(tmp, "w") as f:
        f.write(built_for)
    os.replace(tmp, BINDING_FOR)
    return BINDING


def build(force: bool = False, verbose: bool = False) -> str:
    lib = build_library(force, verbose)
    build_binding(force, verbose)
    return lib


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        return LIB
    nvcc = nvcc_path()
    objdir = os.path.join(ROOT, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    for src in SOURCES:
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        cmd = [nvcc, *nvcc_flags(), "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        objs.append(obj)
    tmp = LIB + ".tmp"
    cmd = [nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs,
           "-cudart", "static"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB)
