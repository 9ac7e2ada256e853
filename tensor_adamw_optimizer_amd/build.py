"""Build step of the HIP library: compiles csrc/*.hip for gfx950 into
``libapexw.so`` next to this file (in-tree, so it travels with the sources).
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
SRC = os.path.join(CSRC, "apexw.hip")
# the operators around the optimizer step, a translation unit each
OP_SRCS = [os.path.join(CSRC, n) for n in ("ops_gated_ffn.hip", "ops_linear_xent.hip",
                                               "ops_qk_norm_rope.hip")]
DEPS = [SRC, *OP_SRCS, os.path.join(ROOT, "include", "apexw.h"),
        *(os.path.join(CSRC, n) for n in ("apexw_kernels.hpp", "apexw_plan.hpp", "ops_common.hpp",
                                          "ops_gemm.hpp", "ops_rounds.hpp", "ops_rows.hpp"))]
LIB = os.path.join(HERE, "libapexw.so")
ARCH = os.environ.get("APEXW_OFFLOAD_ARCH", "gfx950")

BASE_FLAGS = [
    "-O3", "-std=c++17", "-fPIC", "-Wall",
    "--offload-arch=" + ARCH,
    # packed fp32 instructions are not generated
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]
FLAGS = [
    "-shared", *BASE_FLAGS,
    # every fp32 operation separately rounded: no FMA contraction, correctly
    # rounded division and square root, denormals kept
    "-ffp-contract=off", "-fno-fast-math",
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-fno-gpu-flush-denormals-to-zero",
]
# the operators need no such fixed rounding order: their error bounds count
# contracted multiply-adds too
OP_FLAGS = [*BASE_FLAGS, "-fno-gpu-flush-denormals-to-zero"]


def _hipcc(args, verbose: bool) -> None:
    cmd = ["hipcc", *args]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(l for l in res.stdout.splitlines()
                    if "packed-fp32-ops" not in l)   # host pass: unknown feature
    if res.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + out)
    if out.strip() and verbose:
        print(out, flush=True)


def build(verbose: bool = False) -> str:
    """Compiles each translation unit to an object (in parallel) and links
    them into the library."""
    inc = ["-I", os.path.join(ROOT, "include")]
    flags = [f for f in FLAGS if f != "-shared"]
    with tempfile.TemporaryDirectory(prefix="apexw_build_") as tmp, \
            ThreadPoolExecutor(max_workers=4) as pool:
        jobs, objs = [], []
        for src in (SRC, *OP_SRCS):
            obj = os.path.join(tmp, os.path.basename(src) + ".o")
            objs.append(obj)
            jobs.append(pool.submit(_hipcc, [*(flags if src == SRC else OP_FLAGS), *inc, "-c",
                                             "-o", obj, src], verbose))
        for j in jobs:
            j.result()
        out = LIB + ".tmp%d" % os.getpid()
        try:
            _hipcc(["-shared", "-fPIC", "--offload-arch=" + ARCH, "-o", out, *objs], verbose)
            os.replace(out, LIB)
        finally:
            if os.path.exists(out):
                os.remove(out)
    return LIB


RULES = os.path.join(ROOT, "tests", "rules")
CHECKS = [(os.path.join(RULES, src), os.path.join(RULES, lib))
          for src, lib in (("bf16_all.hip", "libbf16_all.so"),
                           ("rcp_sqrt_all.hip", "librcp_sqrt_all.so"))]


def build_checks(verbose: bool = False) -> list:
    """The test-only device checks of the kernel header's conversion,
    square root, reciprocal and short division (tests/rules), each its own
    library (each includes the kernel header), built with the library's
    flags."""
    built = []
    for src, lib in CHECKS:
        tmp = lib + ".tmp%d" % os.getpid()
        cmd = ["hipcc", *FLAGS, "-I", os.path.join(ROOT, "include"), "-I",
               os.path.join(HERE, "csrc"), "-o", tmp, src]
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
        if res.returncode != 0:
            if os.path.exists(tmp):
                os.remove(tmp)
            raise RuntimeError("hipcc failed:\n" + res.stdout)
        os.replace(tmp, lib)
        built.append(lib)
    return built


def is_stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(d) > t for d in DEPS)


if __name__ == "__main__":
    print(build(verbose=True))
    sys.exit(0)
