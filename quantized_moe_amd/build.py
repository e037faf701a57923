"""Build libqmoe.so (the HIP library) in-tree for gfx950, and the Python calls on it.

Each .hip source is compiled separately (the router and gate files with
floating-point contraction off, so their fixed fp32 steps are exactly what the
source says), then linked into one shared library next to this file.
_calls.so, the Python module of the gate and block-scaled operators, is host
code that reads torch tensors and calls that library.
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libqmoe.so")
PROBE_OUT = os.path.join(HERE, "libqmoe_probe.so")  # measurement probes (not the layer's ABI)
CALLS_OUT = os.path.join(HERE, "_calls.so")
OBJ = os.path.join(HERE, "_build")
ARCH = "gfx950"

SOURCES = ["api.hip", "route.hip", "bucket.hip", "repack.hip", "decode.hip", "decode_k1.hip", "decode_k2.hip",
           "decode_k3.hip", "decode_unique.hip", "prefill.hip", "dense.hip", "gate.hip", "blockscale_quant.hip",
           "blockscale_matmul.hip", "blockscale_experts.hip", "int8_quant.hip", "int8_matmul.hip", "int8_experts.hip",
           "balance.hip"]
PROBE_SOURCES = ["probe.hip"]
# packed-fp32 VALU forms are disabled: only ordinary fp32 instructions
COMMON = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-Xclang", "-target-feature", "-Xclang",
          "-packed-fp32-ops", "-I", os.path.join(ROOT, "include"), "-Wall", "-Wno-unused-function"]
PER_FILE = {"route.hip": ["-ffp-contract=off"], "gate.hip": ["-ffp-contract=off"]}
# hipBLASLt runs the dense shared-expert GEMMs of long prefill chunks (dense.hip)
LIBS = ["-L/opt/rocm/lib", "-lhipblaslt"]


def _compile(src: str) -> str:
    obj = os.path.join(OBJ, src.replace(".hip", ".o"))
    cmd = ["hipcc", "-c", os.path.join(CSRC, src), "-o", obj] + COMMON + PER_FILE.get(src, [])
    r = subprocess.run(cmd, capture_output=True, text=True)
    msgs = "\n".join(l for l in (r.stdout + r.stderr).splitlines()
                     if "packed-fp32-ops" not in l and "hip-link" not in l and l.strip())
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{msgs}")
    if msgs:
        print(msgs, file=sys.stderr)
    return obj


def _link(objs, out, libs=()):
    tmp = out + ".tmp"
    cmd = ["hipcc", "-shared", "-o", tmp, f"--offload-arch={ARCH}"] + objs + list(libs)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, out)


def _compile_calls() -> str:
    import torch

    t = os.path.dirname(torch.__file__)
    obj = os.path.join(OBJ, "calls.o")
    cmd = ["g++", "-c", os.path.join(CSRC, "calls.cpp"), "-o", obj, "-O2", "-std=c++17", "-fPIC", "-Wall",
           "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(ROOT, "include"), "-isystem", os.path.join(t, "include"), "-isystem", "/opt/rocm/include",
           "-isystem", sysconfig.get_path("include")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for calls.cpp:\n" + r.stdout + r.stderr)
    return obj


def _link_calls(obj: str) -> None:
    import torch

    tmp = CALLS_OUT + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", HERE, "-l:libqmoe.so", "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, CALLS_OUT)


def build(verbose: bool = True) -> str:
    os.makedirs(OBJ, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(10, os.cpu_count() or 1)) as ex:
        calls = ex.submit(_compile_calls)
        objs = list(ex.map(_compile, SOURCES + PROBE_SOURCES))
    _link(objs[:len(SOURCES)], OUT, LIBS)
    _link(objs[len(SOURCES):], PROBE_OUT)
    _link_calls(calls.result())
    if verbose:
        print(f"built {OUT}, {PROBE_OUT} and {CALLS_OUT}")
    return OUT


if __name__ == "__main__":
    build()
