"""Build libmrope.so (HIP, gfx950) in-tree with hipcc."""
from __future__ import annotations

import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libmrope.so")
OBJ = os.path.join(PKG, "_build")
SOURCES = ["mrope_kernels.hip", "mrope_abi.hip", "mrope_append.hip", "mrope_attend.hip", "mrope_pages.hip",
           "mrope_attend_tree.hip", "mrope_tree.hip", "mrope_verify.hip", "mrope_kv8_abi.hip"]

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-std=c++17",
    "-O3",
    "-fPIC",
    "-shared",
    "-ffp-contract=off",
    # keep the compiler away from packed fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
]


def build(verbose: bool = False) -> str:
    """Compile every source (one hipcc each, in parallel) and link the library."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    os.makedirs(OBJ, exist_ok=True)
    objs = [os.path.join(OBJ, s + ".o") for s in SOURCES]
    inc = ["-I", os.path.join(ROOT, "include"), "-I", CSRC]
    with ThreadPoolExecutor(4) as ex:
        msgs = list(ex.map(lambda so: _run([hipcc, *(f for f in HIPCC_FLAGS if f != "-shared"), *inc, "-c", os.path.join(CSRC, so[0]), "-o", so[1]]),
                           zip(SOURCES, objs)))
    tmp = LIB + ".tmp"
    msgs.append(_run([hipcc, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]))
    if verbose and any(msgs):
        print("\n".join(m for m in msgs if m))
    os.replace(tmp, LIB)
    return LIB


def _run(cmd) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass does not know the packed-fp32 feature and says so; that line is harmless.
    noise = "is not a recognized feature for this target"
    msgs = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if noise not in l and l.strip())
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed ({r.returncode}):\n{msgs}")
    return msgs


if __name__ == "__main__":
    print(build(verbose=True))
