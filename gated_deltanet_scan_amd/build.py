"""Build libgdn.so (HIP kernels + C ABI) for gfx950 with hipcc, in-tree."""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRCS = [os.path.join(PKG, "csrc", "gdn_api.hip"),    # scan kernels and their C ABI
        os.path.join(PKG, "csrc", "gdn_block.hip"),  # block projections (hipBLASLt GEMMs)
        os.path.join(PKG, "csrc", "gdn_norm.hip"),   # layer norm
        os.path.join(PKG, "csrc", "gdn_rotary.hip"), # rotary positions
        os.path.join(PKG, "csrc", "gdn_attn.hip"),   # softmax attention: entry points, fp32 kernels
        os.path.join(PKG, "csrc", "gdn_attn_bf16.hip")]   # its bf16 kernels
LIBS = ["-L/opt/rocm/lib", "-lhipblaslt", "-Wl,-rpath,/opt/rocm/lib"]
SO = os.path.join(PKG, "libgdn.so")

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    # keep the compiler from emitting packed fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def build(verbose: bool = False) -> str:
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    compile_flags = [f for f in HIPCC_FLAGS if f != "-shared"]

    def run(cmd):
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, capture_output=True, text=True)
        # hipcc's host pass does not know the gfx950 feature name; that warning is noise
        noise = "is not a recognized feature for this target"
        err = "\n".join(l for l in r.stderr.splitlines() if noise not in l)
        if r.returncode != 0:
            raise RuntimeError("hipcc failed (%d):\n%s" % (r.returncode, err))
        if err.strip() and verbose:
            print(err, file=sys.stderr)

    tmp = SO + ".tmp%d" % os.getpid()
    with tempfile.TemporaryDirectory() as obj_dir, ThreadPoolExecutor(max_workers=len(SRCS)) as pool:
        objs = [os.path.join(obj_dir, os.path.basename(src) + ".o") for src in SRCS]
        # the sources compile side by side, then link
        list(pool.map(lambda so: run([hipcc, *compile_flags, "-I", os.path.join(ROOT, "include"), "-c", so[0],
                                      "-o", so[1]]), zip(SRCS, objs)))
        run([hipcc, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, *LIBS, "-o", tmp])
    os.replace(tmp, SO)
    return SO


if __name__ == "__main__":
    print(build(verbose=True))
