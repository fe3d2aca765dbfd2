"""Builds the gfx950 HIP library ``libgs_hip.so`` in-tree with hipcc: an object
of each source, several at once, and a link.

Flags:
  --offload-arch=gfx950            MI355X (CDNA4) code objects only
  -ffp-contract=fast-honor-pragmas contraction allowed except where a
                                   ``#pragma clang fp contract(off)`` pins the
                                   evaluation order (the decision path)
  -fhip-fp32-correctly-rounded-divide-sqrt   IEEE fp32 division and sqrt
  -munsafe-fp-atomics              hardware fp32 atomic add in the backward
  -target-feature -packed-fp32-ops no packed fp32 instructions
"""

from __future__ import annotations

import glob
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libgs_hip.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-ffp-contract=fast-honor-pragmas", "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-munsafe-fp-atomics", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function", "-Wno-unused-command-line-argument",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")))


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, capture_output=True, text=True)
    out = "\n".join(l for l in (r.stdout + r.stderr).splitlines()
                    if "packed-fp32-ops" not in l and l.strip())
    if r.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + out)
    if verbose and out:
        print(out, file=sys.stderr)


def build(verbose: bool = False, extra=()) -> str:
    """Compile every source and link one shared library (always recompiles)."""
    tmp = LIB + ".tmp%d" % os.getpid()
    jobs = os.environ.get("MAX_JOBS", "")
    jobs = min(8, jobs.isdecimal() and int(jobs) or os.cpu_count() or 1)
    with tempfile.TemporaryDirectory() as folder:
        def compile_one(src):
            obj = os.path.join(folder, os.path.basename(src) + ".o")
            _run([HIPCC] + FLAGS + list(extra) + ["-c", "-I", INCLUDE, "-I", CSRC, "-o", obj, src], verbose)
            return obj

        # the longest first
        with ThreadPoolExecutor(jobs) as pool:
            objs = list(pool.map(compile_one, sorted(sources(), key=os.path.getsize, reverse=True)))
        _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC"] + list(extra) + ["-o", tmp] + objs, verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
