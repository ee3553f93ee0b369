"""Build libq8narrow.so, and its timeline build libq8narrow_timeline.so,
in-tree with hipcc for gfx950.

Flags: -O3, no fast-math, -ffp-contract=off (every fused multiply-add in the
kernels is written out explicitly), and packed-fp32 instructions disabled.
The timeline build adds -DQ8_TIMELINE (per-wave real-time counter records,
include/q8timeline.h); nothing else differs.  The sources are compiled side by
side, each to an object of its own, and linked.
"""

from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(HERE, "libq8narrow.so")
TIMELINE_LIB_PATH = os.path.join(HERE, "libq8narrow_timeline.so")

# the longest to compile first
SOURCES = ["q8_mx_columns.hip", "q8_matmul.hip", "q8_kv4_attend.hip", "q8_mx_matmul.hip", "q8_mx_prompt.hip",
           "q8_norm.hip", "q8_pack.hip", "q8_rope.hip", "q8_measure.hip", "q8_abi.hip", "q8_noalloc.hip",
           "q8_kv4_rows.hip", "q8_kv4_abi.hip", "q8_mx_rows.hip", "q8_ffn_abi.hip"]
HEADERS = ["q8_internal.h", "q8_measure.h", "q8_kv4_internal.h", "q8_kv4_shares.h",
           "q8_ffn_internal.h", "q8_mx_mfma.h", "q8_mx_plan.h", "q8_lds.h"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-Wno-unused-function",
    "-I", INCLUDE,
    "-I", CSRC,
]


def _filtered(text: str) -> str:
    return "\n".join(
        line for line in text.splitlines()
        # hipcc's host pass does not know the device-only feature flag
        if "packed-fp32-ops" not in line and "is not a recognized feature" not in line)


def _run(cmd: list[str], what: str, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    proc = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    msgs = _filtered(proc.stdout)
    if proc.returncode != 0:
        raise RuntimeError(f"hipcc failed ({proc.returncode}) building {what}:\n{msgs}")
    if verbose and msgs.strip():
        print(msgs, file=sys.stderr)


def _build(libs: list[tuple[str, list[str]]], verbose: bool) -> list[str]:
    """Libraries (path, extra flags), all their objects compiled side by side."""
    with tempfile.TemporaryDirectory() as tmp, ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
        jobs = []
        for s in SOURCES:
            for i, (_, extra) in enumerate(libs):
                obj = os.path.join(tmp, f"{i}_{s}.o")
                cmd = [HIPCC, *FLAGS, *extra, "-c", os.path.join(CSRC, s), "-o", obj]
                jobs.append((i, obj, pool.submit(_run, cmd, s, verbose)))
        for _, _, job in jobs:
            job.result()
        for i, (out, extra) in enumerate(libs):
            objs = [obj for k, obj, _ in jobs if k == i]
            _run([HIPCC, *FLAGS, *extra, "-shared", "-o", out + ".tmp", *objs], out, verbose)
            os.replace(out + ".tmp", out)
    return [out for out, _ in libs]


def build(out: str = LIB_PATH, extra_flags: list[str] | None = None,
          verbose: bool = False) -> str:
    """Compile every source into one shared library at ``out``."""
    return _build([(out, list(extra_flags or []))], verbose)[0]


def build_all(verbose: bool = False) -> list[str]:
    """The product library and its timeline build."""
    return _build([(LIB_PATH, []), (TIMELINE_LIB_PATH, ["-DQ8_TIMELINE"])], verbose)


if __name__ == "__main__":
    print("\n".join(build_all(verbose=True)))
