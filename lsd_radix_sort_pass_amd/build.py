"""Build librs.so (the gfx950 HIP library behind include/rs.h) in-tree.

    python -m lsd_radix_sort_pass_amd.build [--save-temps DIR]

Always recompiles.  The library is written to lsd_radix_sort_pass_amd/librs.so.
"""
from __future__ import annotations

import argparse
import os
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "librs.so")
SOURCES = [os.path.join(CSRC, "rs.hip"), os.path.join(CSRC, "experts.hip")]
ARCH = "gfx950"

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    # Packed FP32 instructions are kept out of every code object.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", "hipcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "hipcc"


def build(save_temps: str | None = None, verbose: bool = False) -> str:
    out_tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as objects:
        cwd = PKG
        extra = []
        if save_temps:
            os.makedirs(save_temps, exist_ok=True)
            extra = ["-save-temps"]
            cwd = save_temps
        # One object per source, compiled side by side, then linked.
        jobs, objs = [], []
        for source in SOURCES:
            obj = os.path.join(objects, os.path.basename(source) + ".o")
            cmd = [hipcc(), *extra, *HIPCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", "-o", obj, source]
            if verbose:
                print(" ".join(cmd), flush=True)
            jobs.append((cmd, subprocess.Popen(cmd, cwd=cwd)))
            objs.append(obj)
        codes = [(cmd, job.wait()) for cmd, job in jobs]
        for cmd, code in codes:
            if code != 0:
                raise subprocess.CalledProcessError(code, cmd)
        link = [hipcc(), f"--offload-arch={ARCH}", "-fPIC", "-shared", "-o", out_tmp, *objs]
        if verbose:
            print(" ".join(link), flush=True)
        subprocess.run(link, check=True, cwd=PKG)
    os.replace(out_tmp, LIB)
    return LIB


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--save-temps", default=None, help="keep intermediate files (ISA) in this directory")
    args = ap.parse_args(argv)
    path = build(args.save_temps, verbose=True)
    print(path)
    return 0


if __name__ == "__main__":
    sys.exit(main())
