"""Build libkda.so in-tree with hipcc for gfx950.

Every ``csrc/*.hip`` file is compiled to an object in ``_build/`` (in
parallel), then linked into ``gated_delta_rule_64_amd/libkda.so``.
"""

from __future__ import annotations

import glob
import os
import re
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libkda.so")
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall",
    # no packed fp32 arithmetic in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]

# Sources whose kernels hold every value in registers.  One that spills is
# refused: an earlier form of the fp32 gradients at 192 channels spilled and gave
# wrong sums, for a reason that was not found.
NO_SPILL = ("kda_attn_", "kda_cache")
REMARKS = "-Rpass-analysis=kernel-resource-usage"


def spilling(remarks: str) -> list:
    """The kernels that keep vector registers in memory, by the compiler's
    resource remarks ("name: registers, bytes a lane")."""
    found, name = [], "?"
    spilled = scratch = 0
    for line in remarks.splitlines():
        if m := re.search(r"remark:.*Function Name: (\S+)", line):
            name, spilled, scratch = m.group(1), 0, 0
        elif m := re.search(r"remark:.*ScratchSize \[bytes/lane\]: (\d+)", line):
            scratch = int(m.group(1))
        elif m := re.search(r"remark:.*VGPRs Spill: (\d+)", line):
            spilled = int(m.group(1))
            if spilled or scratch:
                found.append(f"{name}: {spilled}, {scratch}")
    return found


def _hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    cand = os.path.join(rocm, "bin", "hipcc")
    return cand if os.path.exists(cand) else "hipcc"


def _headers_mtime() -> float:
    hdrs = glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(ROOT, "include", "*.h"))
    return max((os.path.getmtime(h) for h in hdrs), default=0.0)


def _compile(src: str, force: bool = True) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    if not force and os.path.exists(obj) and \
            os.path.getmtime(obj) > max(os.path.getmtime(src), _headers_mtime()):
        return obj
    watched = os.path.basename(src).startswith(NO_SPILL)
    cmd = [_hipcc(), *FLAGS, *([REMARKS] if watched else []), "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if watched:
        found = spilling(r.stderr)
        if found or "VGPRs Spill" not in r.stderr:
            os.unlink(obj)  # so that the next build does not take it for a good one
            raise RuntimeError(f"{src}: registers in memory (or no resource remarks):\n" + "\n".join(found))
    return obj


def build(verbose: bool = False, jobs: int = 8, force: bool = True) -> str:
    """Compile and link libkda.so.  force=False reuses objects that are newer
    than their source and every header (for quick rebuilds while editing)."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.hip")))
    with ThreadPoolExecutor(max(1, jobs)) as ex:
        objs = list(ex.map(lambda s: _compile(s, force), srcs))
    tmp = LIB + ".tmp"
    # --no-undefined: a symbol left undefined (e.g. a kernel whose host-side
    # launch stub was not emitted) fails the build here, not at load time
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-Wl,--no-undefined", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    build(verbose=True, force="--changed" not in sys.argv)
