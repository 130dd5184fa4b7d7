"""Build libikbo.so (HIP C++ for gfx950) in-tree with hipcc, and _ikbo_torch.so, the host-side binding
of the cached user histories to torch tensors, with the host compiler.  The library does not need torch: where torch
cannot be imported, it is built alone.

    python -m broadcast_gemm_amd.build
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libikbo.so")
TORCH_LIB = os.path.join(HERE, "_ikbo_torch.so")
SOURCES = ["ikbo_api.cpp", "lce_kernels.hip", "lce_fused.hip", "lce_rows.hip", "lce_stream.hip", "lce_noalloc.hip", "lce_backward.hip", "ikbo_fa.cpp",
           "fa_kernels.hip", "ikbo_history.cpp", "hist_tables.hip", "hist_rope.hip", "hist_cache.hip", "hist_attention.hip"]
ARCH = os.environ.get("IKBO_OFFLOAD_ARCH", "gfx950")


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def torch_command(out: str) -> list:
    """The host compiler's command for the torch binding."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    if not cxx:
        raise RuntimeError("no host C++ compiler")
    include = cpp_extension.include_paths() + [sysconfig.get_paths()["include"], os.path.join(ROOT, "include")]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    return ([cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"]
            + [x for i in include for x in ("-isystem", i)] + [os.path.join(CSRC, "torch_history.cpp"), "-o", out, "-L" + lib]
            + ["-Wl,-rpath," + lib, "-ltorch", "-ltorch_cpu", "-lc10", "-ltorch_python"])


def build(verbose: bool = False) -> str:
    """Compile every HIP/C++ source and link libikbo.so, then the torch binding if torch is there (always rebuilds)."""
    out_dir = os.path.join(ROOT, "_build")
    os.makedirs(out_dir, exist_ok=True)
    common = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-I", os.path.join(ROOT, "include"),
              "-I", CSRC, "-Wall", "-Wno-unused-function",
              # Packed fp32 VALU forms stay off in generated code.
              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
    jobs = []
    for src in SOURCES:
        obj = os.path.join(out_dir, src + ".o")
        cmd = [hipcc()] + common + ["-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        jobs.append((src, obj, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)))
    torch_tmp = TORCH_LIB + ".tmp"
    torch_proc = trouble = None   # the library is linked before any trouble with the binding is raised
    try:
        cmd = torch_command(torch_tmp)
        if verbose:
            print(" ".join(cmd), flush=True)
        torch_proc = subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)
    except Exception as e:
        trouble = e
    objs = []
    for src, obj, proc in jobs:
        _, err = proc.communicate()
        msgs = "\n".join(l for l in (err or "").splitlines() if "packed-fp32-ops" not in l)
        if proc.returncode != 0:
            raise RuntimeError(f"hipcc failed on {src}:\n{msgs}")
        if verbose and msgs.strip():
            print(msgs)
        objs.append(obj)
    tmp = LIB + ".tmp"
    cmd = [hipcc(), "-shared", "-fPIC", f"--offload-arch={ARCH}", "-o", tmp] + objs
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    if isinstance(trouble, ImportError):
        print(f"torch cannot be imported ({trouble}): {os.path.basename(TORCH_LIB)} is not built", file=sys.stderr)
        return LIB
    if trouble is not None:
        raise trouble
    _, err = torch_proc.communicate()
    if torch_proc.returncode != 0:
        raise RuntimeError(f"the host compiler failed on torch_history.cpp:\n{err}")
    os.replace(torch_tmp, TORCH_LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
