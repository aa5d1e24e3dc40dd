"""Build the sm_100a shared library ``libla_pbd.so`` in-tree with nvcc, and with the host compiler
the module ``_la_torch.so`` that binds its operators to torch tensors.

    python -m block_masked_window_b200.build

Every kernel is compiled for ``sm_100a`` only (``-gencode arch=compute_100a,code=sm_100a``)
with ``-lineinfo`` so that profiles map back to source. The CUDA runtime is linked
statically; the CUDA driver is reached at run time through the runtime's entry-point query,
so the library needs no libcuda at link time and builds on a machine without a GPU.
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libla_pbd.so")
BINDING = os.path.join(PKG, "_la_torch.so")
BINDING_SOURCE = os.path.join(CSRC, "torch_binding.cpp")
SOURCES = ["la_pbd_api.cu", "kv_append.cu", "attn_simt.cu", "attn_tc.cu", "combine.cu",
           "la_pbd_static.cu", "prefill_tc.cu", "noop.cu", "la_cache_api.cu", "rope.cu",
           "key_weights.cu", "kv_evict.cu", "verify.cu"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    raise RuntimeError("nvcc not found")


def command(out: str = LIB, extra=None):
    cmd = [nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3",
           "-std=c++17", "--threads", "0", "-Xcompiler", "-fPIC", "-shared", "-Xptxas", "-v",
           "-I", os.path.join(ROOT, "include"), "-o", out]
    cmd += list(extra or [])
    cmd += [os.path.join(CSRC, s) for s in SOURCES]
    return cmd


def binding_command(out: str = BINDING):
    """The module over torch tensors: links the library beside it and torch's own libraries."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) if os.path.sep in nvcc() else "/usr/local/cuda"
    inc = [os.path.join(ROOT, "include"), sysconfig.get_paths()["include"], os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"]
    for d in inc:
        cmd += ["-isystem" if d.startswith(root) else "-I", d]
    return cmd + ["-o", out, BINDING_SOURCE, "-L", PKG, "-l:libla_pbd.so",
                  "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu",
                  "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]


def _make(target, deps, command, verbose):
    """Runs `command` for a temporary file beside `target` if that is older than a dependency."""
    if os.path.exists(target) and os.path.getmtime(target) >= max(os.path.getmtime(d) for d in deps):
        return
    tmp = target + ".tmp"
    res = subprocess.run(command(tmp), capture_output=True, text=True)
    if verbose or res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
    if res.returncode != 0:
        raise RuntimeError(f"building {os.path.basename(target)} failed with exit code {res.returncode}")
    os.replace(tmp, target)


def build(verbose: bool = False) -> str:
    header = os.path.join(ROOT, "include", "la_pbd.h")
    own = [header, os.path.abspath(__file__)]
    deps = [os.path.join(CSRC, s) for s in SOURCES]
    deps += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    _make(LIB, deps + own, command, verbose)
    _make(BINDING, [BINDING_SOURCE] + own, binding_command, verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
