"""Builds the in-tree CUDA libraries for sm_103a with nvcc.

libmoe.so        the engine (csrc/moe_abi.cu, moe_spec.cu, moe_latent.cu, moe_pages.cu and the kernels
                 they include)
libmoe_synth.so  the device twin of the synthetic-input generator

The sources are compiled in parallel, one -gencode (compute_103a / sm_103a),
-O3, -lineinfo, no fast-math, and each library linked from its objects; a
library is rebuilt when a source or header is newer than it.
"""
from __future__ import annotations

import glob
import os
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")

LIBMOE = os.path.join(PKG, "libmoe.so")
LIBSYNTH = os.path.join(PKG, "libmoe_synth.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC"]
LINK = ["-shared", "-Xcompiler", "-fPIC", "-cudart", "static"]


def _nvcc() -> str:
    for p in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc"):
        if p and os.path.exists(p):
            return p
    return "nvcc"


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def targets():
    hdrs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return [
        (LIBMOE, [os.path.join(CSRC, f) for f in ("moe_abi.cu", "moe_spec.cu", "moe_latent.cu", "moe_pages.cu")], hdrs),
        (LIBSYNTH, [os.path.join(CSRC, "moe_synth.cu")], [os.path.join(INCLUDE, "moe_synth.h")]),
    ]


def _run(cmds):
    """Runs the commands in parallel; the failed ones' output."""
    procs = [(c, subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)) for c in cmds]
    logs = [(c, p.communicate()[0], p.returncode) for c, p in procs]
    return [f"{' '.join(c)}\n{log}" for c, log, rc in logs if rc != 0]


def build(force: bool = False, extra_flags=()) -> list:
    """Compile every stale library; returns the list of library paths."""
    stale = [t for t in targets() if force or _stale(t[0], t[1] + t[2])]
    nvcc, pid = _nvcc(), os.getpid()
    compiles, links, objects, moves = [], [], [], []
    for out, srcs, _ in stale:
        objs = [f"{out}.{os.path.basename(s)}.tmp{pid}.o" for s in srcs]
        objects += objs
        compiles += [[nvcc] + ARCH + FLAGS + list(extra_flags) + ["-c", "-o", o, s] for s, o in zip(srcs, objs)]
        tmp = out + f".tmp{pid}"
        links.append([nvcc] + ARCH + LINK + ["-o", tmp] + objs)
        moves.append((tmp, out))
    try:
        errors = _run(compiles) or _run(links)
        if errors:
            raise RuntimeError("nvcc failed:\n" + "\n".join(errors))
        for tmp, out in moves:
            os.replace(tmp, out)
    finally:
        for o in objects:
            if os.path.exists(o):
                os.unlink(o)
    return [t[0] for t in targets()]


if __name__ == "__main__":
    print(build(force=True))
