"""Build libdflash2.so (HIP, gfx950) in-tree with hipcc.

    python -m draft_selection_topk16_amd.build
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SOURCES = [os.path.join(PKG, "csrc", f) for f in ("dflash2.hip", "target.hip", "steps.hip", "fp4.hip")]
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libdflash2.so")
ARCH = "gfx950"


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found")


def compile_flags():
    return [
        f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
        "-I", INCLUDE, "-I", os.path.join(PKG, "csrc"),
        # never emit packed fp32 arithmetic
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-Wno-unused-command-line-argument",
    ]


def build(verbose: bool = False) -> str:
    """Compile the HIP library (its sources side by side, then one link);
    always recompiles."""
    tag = ".tmp%d" % os.getpid()
    objs = [src + tag + ".o" for src in SOURCES]
    cmds = [[hipcc()] + compile_flags() + ["-c", src, "-o", obj] for src, obj in zip(SOURCES, objs)]
    link = [hipcc(), f"--offload-arch={ARCH}", "-fPIC", "-shared"] + objs + ["-o", LIB + tag]
    try:
        if verbose:
            for cmd in cmds:
                print(" ".join(cmd), flush=True)
        running = [subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for cmd in cmds]
        said = [p.communicate()[0] for p in running]
        if all(p.returncode == 0 for p in running):
            if verbose:
                print(" ".join(link), flush=True)
            res = subprocess.run(link, capture_output=True, text=True)
            if res.returncode == 0:
                os.replace(LIB + tag, LIB)
                return LIB
            said.append(res.stdout + res.stderr)
        sys.stderr.write("".join(said))
        raise RuntimeError("hipcc failed building libdflash2.so")
    finally:
        for f in objs + [LIB + tag]:
            if os.path.exists(f):
                os.remove(f)


if __name__ == "__main__":
    print(build(verbose=True))
