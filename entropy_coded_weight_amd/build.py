"""Build the C-ABI library libecw.so in-tree for gfx950 (hipcc; host part with g++)."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libecw.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

# -amdgpu-kernarg-preload-count: the first 11 dwords of kernel arguments arrive in
# scalar registers (k_decode's block-to-tensor fields); code objects keep a
# load-based entry for firmware without preloading.
HIP_FLAGS = [f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-mcode-object-version=5", "-mllvm", "-amdgpu-kernarg-preload-count=11", "-Wall", "-Wno-unused-result",
             f"-I{ROOT}"]
# the torch bindings, of the 4-bit calls and (_fp8.so next to it) of the 8-bit calls, the norm and
# the rotary positions: host code against torch's headers
BIND = os.path.join(HERE, "_mx4.so")


def _bind_flags():
    """Compiler and linker arguments of the binding, or the header that is missing for it."""
    import torch
    from torch.utils.cpp_extension import include_paths
    python, rocm = sysconfig.get_paths()["include"], f"{os.environ.get('ROCM_PATH', '/opt/rocm')}/include"
    dirs = [python, rocm, *include_paths()]
    for header in ("Python.h", "hip/hip_runtime.h", "torch/csrc/autograd/python_variable.h"):
        if not any(os.path.exists(os.path.join(d, header)) for d in dirs):
            return header
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    return (["-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
             "-D__HIP_PLATFORM_AMD__=1", f"-I{python}", f"-I{rocm}"]
            + [f"-isystem{p}" for p in include_paths()],
            [f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip", "-ltorch_hip"])


HIP_SOURCES = ("ecw_kernels.hip", "ecw_probes.hip", "mx4_quant.hip", "mx4_gemm.hip", "kv4.hip", "fp8_quant.hip",
               "fp8_gemm.hip", "rms_norm.hip", "rotary.hip")
HOST_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-Wall", "-Wextra", f"-I{ROOT}"]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"build step failed: {cmd[0]} ... ({r.returncode})")
    if verbose and r.stderr.strip():
        sys.stderr.write(r.stderr)


def build(verbose: bool = False) -> str:
    bdir = os.path.join(HERE, "_build")
    os.makedirs(bdir, exist_ok=True)
    host_o = os.path.join(bdir, "ecw_host.o")
    _run(["g++", *HOST_FLAGS, "-c", os.path.join(CSRC, "ecw_host.cpp"), "-o", host_o], verbose)
    def hip(src):
        obj = os.path.join(bdir, src.replace(".hip", ".o"))
        _run([HIPCC, *HIP_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj], verbose)
        return obj

    with ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
        objs = [host_o, *pool.map(hip, HIP_SOURCES)]
    tmp = LIB + ".tmp"
    _run([HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs, "-lpthread"], verbose)
    os.replace(tmp, LIB)
    found = _bind_flags()
    binds = [(BIND, "mx4_bind.cpp"), (os.path.join(os.path.dirname(BIND), "_fp8.so"), "fp8_bind.cpp")]
    if isinstance(found, str):  # libecw.so does without them; the calls from Python say what is missing
        for bind, _ in binds:
            if os.path.exists(bind):
                os.remove(bind)  # of another state of the sources
            sys.stderr.write(f"{bind} not built: {found} not found; its calls from Python need it\n")
        return LIB
    flags, libs = found
    for bind, src in binds:
        _run(["g++", *flags, os.path.join(CSRC, src), "-o", bind + ".tmp", *libs], verbose)
        os.replace(bind + ".tmp", bind)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
