"""Build ``libtf_ulysses.so`` (in-tree) with nvcc for sm_103a.

The translation units (kernels, host ABI) compile in parallel into
``_build/`` and link into ``ulysses_sequence_attention_tf_gb300/libtf_ulysses.so``;
``_torch_calls.so`` beside it marshals the attention and cache calls.
cudart is linked statically, so the library depends only on the driver.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libtf_ulysses.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
              f"-I{INCLUDE}", f"-I{CSRC}"]
SOURCES = ["block_kernels.cu", "block_kernels_v16.cu", "gemm_kernels.cu", "relayout_kernels.cu", "staged_kernels.cu",
           "tf_ulysses.cpp", "noalloc.cu", "attention_plan.cu", "attention_forward.cu", "attention_backward.cu", "attention_join.cu", "tf_attention.cpp", "kv_append.cu", "kv_attend.cu", "kv_attend_tiles.cu",
           "tf_kv_cache.cpp"]
DEPS = SOURCES + ["relayout.h", "noalloc.h", "device_common.cuh", "block_kernel.cuh", "tma_plan.h", "gemm.h", "host.h",
                  "attention.h", "attention_common.cuh", "attention_order.h", "attention_plan.h",
                  "tcgen05.cuh", "kv_cache.h", "kv_common.cuh"]


# The Python module that marshals the attention and cache calls: C++ against the installed torch.
CALLS_SOURCE = os.path.join(CSRC, "torch_calls.cpp")
CALLS = os.path.join(PKG, "_torch_calls.so")
CALLS_MADE_FOR = os.path.join(BUILD_DIR, "torch_calls_made_for.txt")


def _calls_command(out: str) -> list[str]:
    import sysconfig

    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], INCLUDE]
    return [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-I{d}" for d in include], CALLS_SOURCE, "-o", out,
            f"-L{os.path.join(root, 'lib')}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10"]


def _calls_made_for() -> str:
    """What the module is compiled against beside its sources."""
    import torch
    return f"Python {sys.version}\ntorch {torch.__version__}\n{' '.join(_calls_command('module'))}\n"


def _calls_stale() -> bool:
    if not os.path.exists(CALLS) or not os.path.exists(CALLS_MADE_FOR):
        return True
    with open(CALLS_MADE_FOR) as f:
        if f.read() != _calls_made_for():
            return True
    t = os.path.getmtime(CALLS)
    return any(os.path.getmtime(d) > t for d in (CALLS_SOURCE, os.path.join(INCLUDE, "tf_ulysses.h")))


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, d) for d in DEPS] + [os.path.join(INCLUDE, "tf_ulysses.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def _finish_calls(calls, tmp: str, verbose: bool) -> None:
    cmd, p = calls
    text, _ = p.communicate()
    if verbose or p.returncode != 0:
        sys.stderr.write(text)
    if p.returncode != 0:
        raise RuntimeError("g++ failed:\n" + " ".join(cmd))
    os.replace(tmp, CALLS)
    os.makedirs(BUILD_DIR, exist_ok=True)
    with open(CALLS_MADE_FOR, "w") as f:
        f.write(_calls_made_for())


def build(force: bool = False, verbose: bool = False, defines=(), out: str | None = None) -> str:
    """Compile the library if it is missing or older than its sources.

    ``defines``: extra ``-D`` macros (tuning constants); ``out``: library path
    (default: the in-tree ``libtf_ulysses.so``)."""
    lib = out or LIB
    calls = None  # the in-tree module goes with the in-tree library
    if out is None and (force or _calls_stale()):
        tmp_calls = CALLS + f".tmp{os.getpid()}"
        cmd = _calls_command(tmp_calls)
        calls = (cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))
    if not force and not defines and out is None and not _stale():
        if calls is not None:
            _finish_calls(calls, tmp_calls, verbose)
        return LIB
    build_dir = BUILD_DIR if out is None else os.path.join(os.path.dirname(lib), "_obj")
    os.makedirs(build_dir, exist_ok=True)
    cc = nvcc()
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(build_dir, src + ".o")
        objs.append(obj)
        cmd = [cc, *ARCH, *NVCC_FLAGS, *[f"-D{d}" for d in defines], "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    failed = []
    for cmd, p in procs:
        out, _ = p.communicate()
        if verbose or p.returncode != 0:
            sys.stderr.write(out)
        if p.returncode != 0:
            failed.append(" ".join(cmd))
    if failed:
        raise RuntimeError("nvcc failed:\n" + "\n".join(failed))
    if calls is not None:
        _finish_calls(calls, tmp_calls, verbose)
    tmp = lib + f".tmp{os.getpid()}"
    subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], check=True)
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
