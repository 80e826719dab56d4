"""Builds libmds.so (the HIP kernels and the C-ABI layer) for gfx950 in-tree.

    python -m markov_draft_sampling_amd.build

Each source is compiled by hipcc in parallel, then linked into a shared
library next to this file. Packed fp32 instructions are disabled for device
code. The binding's compiled calls (csrc/calls.cpp, against torch's headers)
become the module _calls beside it.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmds.so")
CALLS = os.path.join(HERE, "_calls.so")
SOURCES = ("abi.hip", "abi_layer.hip", "abi_serve.hip", "draft.hip", "draft_wave.hip", "draft_topk.hip", "kv_cache.hip", "lm_head.hip",
           "lm_head_fp8.hip", "lm_head_mxfp4.hip", "paged_attention.hip", "rope.hip", "verify.hip", "topp.hip")
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    "-Wno-unused-function",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _hipcc() -> str:
    exe = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(exe):
        raise RuntimeError("hipcc not found; the HIP library cannot be built")
    return exe


def _calls_command(out: str):
    """How the module of the binding's compiled calls is built."""
    import importlib.util
    import sysconfig
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    include = os.path.join(torch, "include")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-shared", "-o", out, os.path.join(CSRC, "calls.cpp"),
            "-isystem", include, "-isystem", os.path.join(include, "torch", "csrc", "api", "include"),
            "-isystem", sysconfig.get_paths()["include"], "-L", HERE, "-L", os.path.join(torch, "lib"), "-l:libmds.so",
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-Wl,-rpath,$ORIGIN"]


def build(verbose: bool = False) -> str:
    """Compile every source, link libmds.so and the module of calls; returns the library's path."""
    hipcc = _hipcc()
    os.makedirs(BUILD, exist_ok=True)
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD, src.replace(".hip", ".o"))
        objs.append(obj)
        cmd = [hipcc, *FLAGS, "-I", os.path.join(HERE, "..", "include"), "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    errors = []
    for src, p in procs:
        out, _ = p.communicate()
        out = "\n".join(l for l in out.splitlines() if "packed-fp32-ops" not in l)
        if p.returncode != 0:
            errors.append(f"{src}:\n{out}")
        elif verbose and out.strip():
            print(out)
    if errors:
        raise RuntimeError("hipcc failed:\n" + "\n".join(errors))
    tmp = LIB + ".tmp"
    cmd = [hipcc, f"--offload-arch={ARCH}", "-shared", "-Wl,--no-undefined", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, LIB)
    cmd = _calls_command(CALLS + ".tmp")
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("building the binding's calls failed:\n" + r.stdout + r.stderr)
    os.replace(CALLS + ".tmp", CALLS)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
