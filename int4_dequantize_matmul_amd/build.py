"""Build libq4.so in-tree: hipcc for the gfx950 kernels, g++ for host code.

    python -m int4_dequantize_matmul_amd.build
    python int4_dequantize_matmul_amd/build.py      (the same, without the package)

Where torch can be imported, g++ also compiles the Python binding's small-call
path against its headers (lib/q4_torch.so); libq4.so needs neither torch nor
Python.

Every HIP file is compiled with -ffp-contract=off (no implicit FMA) and
with the packed-FP32 instructions switched off; the host quantizers are
plain C++ so that they also build under the sanitizers (tests/test_host_sanitizers.py
builds them with g++ -fsanitize=address,undefined and drives them over edge
shapes and values).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libq4.so")
TORCH_LIB = os.path.join(LIBDIR, "q4_torch.so")      # the Python binding's small-call path
PROBE_LIB = os.path.join(LIBDIR, "libq4_probe.so")   # the benchmark's ceilings (not the linear)
BUILD = os.path.join(PKG, "_build")
ARCH = "gfx950"

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
HIP_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-result", f"-I{INCLUDE}",
]
# Results of 16 or 32 rows live in vectors of up to 16 registers over a kernel's
# loop; taken apart at the loop's head, each step copied them (64 moves of a
# wave's about 250 other vector instructions).
WHOLE_VECTORS = ["-mllvm", "-amdgpu-codegenprepare-break-large-phis=false"]
FILE_FLAGS = {"attention.hip": WHOLE_VECTORS, "attention_tiled.hip": WHOLE_VECTORS}
CXX_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-ffp-contract=off", "-Wall", "-Wextra", f"-I{INCLUDE}"]


def _run(cmd):
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(l for l in r.stdout.splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"build step failed: {' '.join(cmd)}\n{out}")
    return out


def _torch_binding(out: str) -> list | None:
    """The compile of csrc/binding/q4_torch.cpp against the installed torch, if there is one."""
    import sysconfig

    try:
        import torch
    except ImportError:
        return None
    root = os.path.dirname(torch.__file__)
    inc = [sysconfig.get_paths()["include"], os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include")]
    return ["g++", *CXX_FLAGS, "-Wno-unused-parameter", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *(f"-isystem{i}" for i in inc), "-shared", "-o", out, os.path.join(CSRC, "binding", "q4_torch.cpp"),
            f"-L{os.path.join(root, 'lib')}", "-lc10", "-ltorch_cpu", "-ltorch_python"]


def build(verbose: bool = False) -> str:
    """Compile every source and link lib/libq4.so; returns the library path."""
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    jobs = []
    for src in sorted(glob.glob(os.path.join(CSRC, "*.hip"))):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        jobs.append([HIPCC, *HIP_FLAGS, *FILE_FLAGS.get(os.path.basename(src), []), "-c", src, "-o", obj])
    for src in sorted(glob.glob(os.path.join(CSRC, "*.cpp"))):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        jobs.append(["g++", *CXX_FLAGS, "-c", src, "-o", obj])
    objs = [j[-1] for j in jobs]
    binding = _torch_binding(TORCH_LIB + ".tmp")
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        results = [ex.submit(_run, j) for j in jobs]
        bound = ex.submit(_run, binding) if binding else None
        for r in results:
            out = r.result()
            if verbose and out.strip():
                print(out)
        tmp = LIB + ".tmp"
        _run([HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs])
        os.replace(tmp, LIB)
        probe_src = os.path.join(CSRC, "probe", "q4_probe.hip")
        tmp = PROBE_LIB + ".tmp"
        _run([HIPCC, *HIP_FLAGS, "-shared", "-o", tmp, probe_src])
        os.replace(tmp, PROBE_LIB)
        if bound:
            bound.result()
            os.replace(TORCH_LIB + ".tmp", TORCH_LIB)
        else:
            print("no torch: libq4.so is built, the Python binding's lib/q4_torch.so is not")
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
