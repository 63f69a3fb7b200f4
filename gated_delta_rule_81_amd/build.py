"""Build ``libkda.so`` (the C-ABI library of include/kda.h) with hipcc for gfx950.

Usage:  python -m gated_delta_rule_81_amd.build   (or ``build()`` from Python)

Every HIP source is compiled separately (in parallel) and linked into one
shared library next to this file; beside it the CPython module ``_cache_calls.so``
(csrc/py_cache.cpp, host code on torch's headers).  Flags:
  --offload-arch=gfx950       MI355X only
  -packed-fp32-ops (disabled) keep the compiler from emitting packed fp32 ops
  -mcode-object-version=5     loadable by the HIP runtime PyTorch bundles
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libkda.so")
CALLS = os.path.join(HERE, "_cache_calls.so")

SOURCES = ["kda_api.cpp", "kda_decode.hip", "kda_chunk.hip", "kda_seq.hip", "kda_segment.hip",
           "kda_bwd.hip", "kda_bwd_chain.hip", "layer_api.cpp", "conv.hip", "qk_norm.hip",
           "ssm_scan.hip", "ssm_step.hip", "ssm_bwd.hip", "cache_api.cpp", "cache_append.hip",
           "attn.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
         "-mcode-object-version=5",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wall", "-Wno-unused-function",
         "-I", INCLUDE, "-I", CSRC]
# Per-source flags: the pipelined dL/dS chain and the fp32 token recurrences
# (kda_seq.hip) are faster with the machine scheduler that favours
# instruction-level parallelism; the other kernels keep the default, which
# measured faster for them.
_ILP = ["-mllvm", "-amdgpu-sched-strategy=max-ilp"]
SOURCE_FLAGS = {"kda_bwd_chain.hip": _ILP, "kda_seq.hip": _ILP}


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, *SOURCE_FLAGS.get(src, []), "-x", "hip", "-c", os.path.join(CSRC, src),
           "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    # the host pass does not know the packed-fp32 feature name; that is expected
    noise = "is not a recognized feature for this target"
    msgs = [ln for ln in (res.stdout + res.stderr).splitlines() if noise not in ln]
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n" + "\n".join(msgs))
    if verbose and msgs:
        print("\n".join(msgs), file=sys.stderr)
    return obj


def _calls(verbose: bool) -> None:
    """The CPython module.  torch's libraries are found by name when it is imported:
    torch has loaded them by then."""
    import torch
    from torch.utils.cpp_extension import include_paths, library_paths

    paths = [*include_paths(), sysconfig.get_paths()["include"]]
    tmp = CALLS + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[x for p in paths for x in ("-isystem", p)], os.path.join(CSRC, "py_cache.cpp"), "-o", tmp,
           *[f"-L{p}" for p in library_paths()], "-ltorch_python", "-ltorch_cpu", "-lc10"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed for py_cache.cpp:\n" + res.stderr)
    if verbose and res.stderr:
        print(res.stderr, file=sys.stderr)
    os.replace(tmp, CALLS)


def build(verbose: bool = False) -> str:
    """Compile every source and link ``libkda.so``; returns its path.  Where the
    module beside it cannot be built, the library is there all the same, no older module
    is left to call it, and the error is raised."""
    os.makedirs(BUILD, exist_ok=True)
    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as pool:
        calls = pool.submit(_calls, verbose)
        objs = list(pool.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + ".tmp"
    subprocess.run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs],
                   check=True, capture_output=not verbose)
    os.replace(tmp, LIB)
    if calls.exception() is not None:
        if os.path.exists(CALLS):
            os.remove(CALLS)
        raise calls.exception()
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
