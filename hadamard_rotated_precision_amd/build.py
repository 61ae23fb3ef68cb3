"""Build libhq.so (the gfx950 HIP kernels and the C ABI of include/hq.h) and libhq_train.so (those
of include/hq_train.h) in-tree with hipcc."""
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libhq.so")

SOURCES = ["hq_rotate.hip", "hq_prologue.hip", "hq_gemm.hip", "hq_static.hip", "hq_lss.hip", "hq_api.cpp",
           "hq_profile.cpp"]
# the operators of include/hq_train.h, a library of their own that links libhq.so
TRAIN_LIB = os.path.join(HERE, "libhq_train.so")
TRAIN_SOURCES = ["hq_block.hip", "hq_block_gemm.hip", "hq_block_gemv.hip", "hq_adamw.hip",
                 "hq_train_api.cpp"]

# -packed-fp32-ops: hipcc forms packed fp32 ops from plain float code; keep them out.
HIP_FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-Wall", "-Wno-unused-function", "-Wno-unused-variable",
             "-I" + os.path.join(ROOT, "include")]


TRAIN_LINK = ["-L" + HERE, "-lhq", "-Wl,-rpath,$ORIGIN"]


def link(lib, objs, verbose=False, extra=()):
    cmd = (["hipcc", "--offload-arch=gfx950", "-shared", "-fPIC"] + objs + list(extra) +
           ["-o", lib + ".tmp"])
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(lib + ".tmp", lib)


def build(verbose=False, jobs=None):
    objs = []
    procs = []
    for src in SOURCES + TRAIN_SOURCES:
        obj = os.path.join(CSRC, src + ".o")
        lang = ["-x", "hip"] if src.endswith(".hip") else []
        cmd = ["hipcc"] + HIP_FLAGS + lang + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((cmd, subprocess.Popen(cmd)))
        objs.append(obj)
    for cmd, p in procs:
        if p.wait() != 0:
            raise RuntimeError("compile failed: " + " ".join(cmd))
    n = len(SOURCES)
    link(LIB, objs[:n], verbose)
    link(TRAIN_LIB, objs[n:], verbose, TRAIN_LINK)
    for o in objs:
        os.remove(o)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
