"""Build the HIP library libmoe.so for gfx950, in place."""
from __future__ import annotations

import concurrent.futures
import glob
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libmoe.so")

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-result", "-fvisibility=hidden",
]


def sources():
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.hip")))


def build(verbose: bool = False) -> str:
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    out_tmp = LIB + ".tmp"

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("hipcc failed building libmoe.so")

    with tempfile.TemporaryDirectory() as tmp:
        objs = [os.path.join(tmp, os.path.basename(f) + ".o")
                for f in sources()]
        # one compiler a source file, up to 8 at once
        with concurrent.futures.ThreadPoolExecutor(8) as pool:
            list(pool.map(run, [
                [hipcc, *HIPCC_FLAGS, "-c", "-I", os.path.join(ROOT, "include"),
                 "-I", os.path.join(HERE, "csrc"), f, "-o", o]
                for f, o in zip(sources(), objs)]))
        run([hipcc, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o",
             out_tmp])
    os.replace(out_tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
