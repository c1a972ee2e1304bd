"""Builds libwkv7.so (the HIP kernels and the C ABI) in-tree, for gfx950 only."""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB_PATH = os.path.join(PKG, "libwkv7.so")
SOURCES = ["wkv7_api.hip", "wkv7_step.hip", "wkv7_chunk.hip", "wkv7_tail.hip", "wkv7_bwd.hip", "wkv7_bwdc.hip",
           "gdr_api.hip", "gdr_step.hip", "gdr_chain.hip", "gdr_grad.hip", "draft.hip"]
ARCH = "gfx950"

# -packed-fp32-ops: no packed fp32 math is emitted for any kernel of this library.
HIPCC_FLAGS = ["-O3", "-std=c++17", "-fPIC", "-shared", f"--offload-arch={ARCH}",
               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
               "-Wall", "-Wno-unused-function"]


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return os.path.join(rocm, "bin", "hipcc")


def build(verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compile every source (a process each) and link libwkv7.so.  Always recompiles.  Returns the path."""
    flags = [hipcc()] + HIPCC_FLAGS + (extra_flags or []) + ["-I", os.path.join(ROOT, "include")]
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    with tempfile.TemporaryDirectory() as work:
        objs = [os.path.join(work, s + ".o") for s in SOURCES]
        cmds = [[f for f in flags if f != "-shared"] + ["-c", os.path.join(CSRC, s), "-o", o]
                for s, o in zip(SOURCES, objs)]
        with ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
            list(pool.map(lambda c: _run(c, verbose), cmds))
        _run([hipcc(), "-shared", f"--offload-arch={ARCH}"] + objs + ["-o", tmp], verbose)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def _run(cmd: list[str], verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass does not know the packed-fp32 feature and says so; that is harmless.
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in res.stderr.splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{err}")
    if verbose and err.strip():
        print(err, file=sys.stderr)


if __name__ == "__main__":
    print(build(verbose=True))
