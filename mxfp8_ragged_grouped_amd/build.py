"""Build the HIP library in-tree for gfx950.

    python -m mxfp8_ragged_grouped_amd.build

compiles the HIP sources of csrc/ with hipcc, each on its own, and links them
into lib/libmxfp8_wgrad.so (the library the Python binding loads).  Packed-FP32
instruction selection is disabled for all device code.
"""
from concurrent.futures import ThreadPoolExecutor
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SOURCES = [os.path.join(HERE, "csrc", n) for n in ("mxfp8_wgrad.hip", "ortho.hip", "vocab_loss.hip", "moe_layer.hip",
                                                  "tokens.hip", "grad_norm.hip", "linear4.hip")]
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(HERE, "lib")
LIB = os.path.join(LIB_DIR, "libmxfp8_wgrad.so")
ARCH = "gfx950"

HIPCC_FLAGS = [
    "-O3", "-std=c++17", "-fPIC",
    "--offload-arch=" + ARCH,
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def hipcc():
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return os.path.join(rocm, "bin", "hipcc")


def build(verbose=False):
    """Compile the library (always recompiles).  Returns the .so path."""
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp = LIB + ".tmp%d" % os.getpid()
    with tempfile.TemporaryDirectory() as objects:
        outs = [os.path.join(objects, os.path.basename(s) + ".o") for s in SOURCES]
        with ThreadPoolExecutor(4) as pool:
            list(pool.map(lambda a: _run(["-I", INCLUDE, "-c", a[0], "-o", a[1]], verbose), zip(SOURCES, outs)))
        _run(["-shared"] + outs + ["-o", tmp], verbose)
    os.replace(tmp, LIB)
    return LIB


def _run(args, verbose):
    cmd = [hipcc()] + HIPCC_FLAGS + args
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass reports the device-only target feature as unknown: harmless
    err = "\n".join(l for l in res.stderr.splitlines() if "packed-fp32-ops" not in l)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + err)
    if err.strip() and verbose:
        print(err, file=sys.stderr)


if __name__ == "__main__":
    print(build(verbose=True))
