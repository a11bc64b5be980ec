"""Build libecho.so (HIP, gfx950) in-tree with hipcc.

Flags:
  -ffp-contract=off   every a*b+c stays a separate multiply and add, as the
                      method's binary32 operation order requires (the layer
                      operators ask for fused multiply-adds by name);
  -Xclang -target-feature -Xclang -packed-fp32-ops
                      no packed FP32 instructions are generated;
  no fast-math: fp32 division stays correctly rounded, denormals are kept.

Each source is compiled to an object of its own, a few at a time, and the
objects are linked into the library.
"""
import glob
import os
import shutil
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libecho.so")
SOURCES = sorted(glob.glob(os.path.join(HERE, "csrc", "*.hip")))
HIPCC = os.environ.get("HIPCC", shutil.which("hipcc") or "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-ffp-contract=off", "-fno-fast-math",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    "-I", os.path.join(ROOT, "include"), "-I", os.path.join(HERE, "csrc"),
]


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in (r.stderr or "").splitlines() if noise not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed ({r.returncode}):\n{err}")
    if verbose and err.strip():
        print(err)


def build(verbose: bool = False, extra=()) -> str:
    with tempfile.TemporaryDirectory() as tmp:
        objects = [os.path.join(tmp, f"{i}.o") for i in range(len(SOURCES))]
        with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as pool:
            list(pool.map(lambda so: _run([HIPCC, *FLAGS, *extra, "-c", so[0], "-o", so[1]], verbose),
                          zip(SOURCES, objects)))
        linked = LIB + ".tmp"
        _run([HIPCC, f"--offload-arch={ARCH}", "-fPIC", "-shared", *objects, "-o", linked], verbose)
    os.replace(linked, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
