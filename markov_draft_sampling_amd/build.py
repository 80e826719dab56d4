"""Builds libmds.so (the HIP kernels and the C-ABI layer) for gfx950 in-tree.

    python -m markov_draft_sampling_amd.build

Each source is compiled by hipcc in parallel, then linked into a shared
library next to this file. Packed fp32 instructions are disabled for device
code. The binding's compiled calls (csrc/calls.cpp, against torch's headers)
become the module _calls beside it; without torch the library is built alone.
Both are put in place together, once both are built.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmds.so")
CALLS = os.path.join(HERE, "_calls" + sysconfig.get_config_var("EXT_SUFFIX"))  # (for this interpreter alone)
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


def _calls_command(lib: str, out: str):
    """How the module of the binding's compiled calls is built against the library, or None without torch."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    torch = os.path.dirname(spec.origin)
    include = os.path.join(torch, "include")
    cxx = ["g++"] if shutil.which("g++") else [_hipcc(), "-x", "c++", "-no-hip-rt"]
    return [*cxx, "-O2", "-std=c++17", "-fPIC", "-Wall", "-shared", "-o", out, os.path.join(CSRC, "calls.cpp"),
            "-isystem", include, "-isystem", os.path.join(include, "torch", "csrc", "api", "include"),
            "-isystem", sysconfig.get_paths()["include"], "-L", os.path.dirname(lib), "-L", os.path.join(torch, "lib"),
            "-l:libmds.so", "-ltorch_python", "-ltorch_cpu", "-lc10", "-Wl,-rpath,$ORIGIN"]


def _link(cmd, what: str, verbose: bool):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n" + r.stdout + r.stderr)


def _remove(*paths):
    for path in paths:
        if os.path.exists(path):
            os.remove(path)


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
    lib, calls = (os.path.join(BUILD, os.path.basename(path)) for path in (LIB, CALLS))
    try:
        _link([hipcc, f"--offload-arch={ARCH}", "-shared", "-Wl,--no-undefined", "-o", lib, *objs], "link", verbose)
        cmd = _calls_command(lib, calls)
        if cmd:
            _link(cmd, "building the binding's calls", verbose)
        else:
            print("torch is not installed: libmds.so is built alone, without the module of the binding's compiled calls",
                  file=sys.stderr, flush=True)
        # modules of before (of other interpreters too) would call this library by another one's signatures
        _remove(*(set(glob.glob(os.path.join(HERE, "_calls*.so"))) - ({CALLS} if cmd else set())))
        os.replace(lib, LIB)
        if cmd:
            os.replace(calls, CALLS)
    finally:
        _remove(lib, calls)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
