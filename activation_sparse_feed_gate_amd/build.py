"""Build the gfx950 HIP library ``libtw.so`` in-tree with hipcc.

Every HIP source is compiled for gfx950 only, with the packed-fp32 target
feature switched off (the compiler then never emits packed fp32 add/mul/fma),
and linked into one shared library exporting the C ABI of ``include/tw.h``.
``_tw_calls.so``, the native part of the Python binding, is host code compiled
against the installed torch and linked to that library.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIBRARY = os.path.join(HERE, "libtw.so")
CALLS = os.path.join(HERE, "_tw_calls.so")  # native part of the Python binding (csrc/tw_calls.cpp)
PEAK_PROBE = os.path.join(HERE, "peak_probe")  # achievable-peak program (csrc/peak_probe.hip)

SOURCES = ["gate_twell.hip", "pack_dense.hip", "sparse_updown.hip", "dense_ffn.hip", "hybrid.hip",
           "layer_norm.hip", "quant_gemm.hip", "gated_ffn.hip", "linear_ce.hip", "grad_clip.hip",
           "tw_api.cpp"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Wall",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE, "-I", CSRC,
]


def _torch_dir() -> str:
    import importlib.util

    return os.path.dirname(importlib.util.find_spec("torch").origin)


def _calls_flags() -> list:
    inc = os.path.join(_torch_dir(), "include")
    return ["-O2", "-std=c++17", "-fPIC", "-Wall", "-I", INCLUDE, "-isystem", inc, "-isystem",
            os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem",
            sysconfig.get_paths()["include"]]


def build(verbose: bool = False) -> str:
    """Compile all sources (in parallel) and link ``libtw.so`` and, to it,
    ``_tw_calls.so``; returns the library's path.  A failure of the latter alone
    raises with the library built and no older ``_tw_calls.so`` beside it."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    procs = []
    objs = []
    calls_obj = os.path.join(BUILD_DIR, "tw_calls.cpp.o")
    for src in ["tw_calls.cpp"] + SOURCES:
        obj = os.path.join(BUILD_DIR, src + ".o")
        if obj == calls_obj:
            flags = _calls_flags()
        else:
            objs.append(obj)
            flags = FLAGS + (["-x", "hip"] if src.endswith(".cpp") else [])
        cmd = [HIPCC, *flags, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if out and (verbose or p.returncode):
            sys.stderr.write(out.decode(errors="replace"))
        if p.returncode:
            failed.append(src)
    if any(src in SOURCES for src in failed):
        raise RuntimeError(f"hipcc failed for {failed}")
    if os.path.exists(CALLS):  # never an older one beside a newer library
        os.remove(CALLS)
    tmp = LIBRARY + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIBRARY)
    if failed:
        raise RuntimeError(f"hipcc failed for {failed}")
    tmp = CALLS + ".tmp"
    cmd = [HIPCC, "-shared", "-fPIC", calls_obj, "-o", tmp, "-L", HERE, "-l:libtw.so", "-L",
           os.path.join(_torch_dir(), "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch_hip",
           "-lc10", "-lc10_hip", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, CALLS)
    return LIBRARY


def build_peak_probe(verbose: bool = False) -> str:
    """Compile the standalone achievable-peak program (a measurement tool,
    not part of the library: built only on request, with
    ``python -m activation_sparse_feed_gate_amd.build --peak-probe``);
    returns its path."""
    cmd = [HIPCC, *FLAGS, os.path.join(CSRC, "peak_probe.hip"), "-o", PEAK_PROBE]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    return PEAK_PROBE


if __name__ == "__main__":
    if "--peak-probe" in sys.argv:
        print(build_peak_probe(verbose="-v" in sys.argv))
    else:
        print(build(verbose="-v" in sys.argv))
