"""Build ``libbasp.so`` in-tree with hipcc for gfx950 (MI355X).

    python -m sequence_re_layout_amd.build

The library is the product: the HIP kernels and the C ABI declared in
``include/basp.h``.  The Python binding loads it from this directory.
"""
import concurrent.futures
import os
import subprocess
import sys
import tempfile
import time

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libbasp.so")
SOURCES = [os.path.join(CSRC, f) for f in ("plan.cpp", "launch.cpp", "index_plan.cpp", "relayout.hip",
                                           "expert.hip", "embed.hip")]
ARCH = "gfx950"


def hipcc():
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    path = os.path.join(rocm, "bin", "hipcc")
    return path if os.path.exists(path) else "hipcc"


def _run(cmd):
    """stderr of one hipcc command, without what is harmless."""
    res = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass does not know the packed-fp32 feature; that warning is harmless
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in res.stderr.splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + err)
    return err


def build(verbose: bool = False) -> str:
    """Compile every source into libbasp.so (always recompiles): an object per
    source, side by side, and one link."""
    tmp = LIB + ".tmp%d" % os.getpid()
    common = [hipcc(), "--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-command-line-argument",
              # packed fp32 instructions stay off in all device code
              "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I", INCLUDE, "-I", CSRC]
    t0 = time.time()
    with tempfile.TemporaryDirectory(prefix="basp_build_") as d:
        objects = [os.path.join(d, os.path.basename(src) + ".o") for src in SOURCES]
        compiles = [common + ["-c", src, "-o", obj] for src, obj in zip(SOURCES, objects)]
        link = common + ["-shared"] + objects + ["-o", tmp]
        if verbose:
            for cmd in compiles + [link]:
                print(" ".join(cmd), flush=True)
        with concurrent.futures.ThreadPoolExecutor(len(SOURCES)) as pool:
            errs = list(pool.map(_run, compiles))
        errs.append(_run(link))
    if verbose:
        for err in errs:
            if err.strip():
                print(err, file=sys.stderr)
    os.replace(tmp, LIB)
    if verbose:
        print("built %s in %.1f s" % (LIB, time.time() - t0), flush=True)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
