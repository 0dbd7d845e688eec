"""Build libgptq_mi355x.so (gfx950) in-tree with hipcc.

    python -m post_weight_quantization_18_amd.build [--debug]

--debug builds libgptq_mi355x_debug.so instead: -DGPTQ_DEBUG turns on the
device-side bounds checks (GPTQ_DASSERT), objects under _build/debug/. The
binding loads it when GPTQ_MI355X_LIB names it.

Each .hip source is compiled to an object under _build/ (in parallel) and the
objects are linked into post_weight_quantization_18_amd/libgptq_mi355x.so.
Packed fp32 instructions are disabled on purpose (-packed-fp32-ops).
"""

from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libgptq_mi355x.so")
LIB_DEBUG = os.path.join(PKG, "libgptq_mi355x_debug.so")
SOURCES = ["gptq_api.hip", "syrk.hip", "chain.hip", "quant.hip", "trail.hip", "order.hip", "gemv.hip", "trace.hip",
           "kv_cache.hip", "kv_token.hip", "kv_prompt.hip",
           "colloop_row.hip", "colloop_g16.hip", "colloop_g32.hip", "colloop_g64.hip", "colloop_g128.hip", "colloop_wide.hip",
           "colloop_static.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
FLAGS = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wno-unused-result", "-Werror=inline-asm", "-I", os.path.join(ROOT, "include")]


def _run(cmd):
    p = subprocess.run(cmd, capture_output=True, text=True)
    out = "\n".join(l for l in (p.stdout + p.stderr).splitlines()
                    if "packed-fp32-ops" not in l)
    if p.returncode != 0:
        raise RuntimeError(f"command failed ({p.returncode}): {' '.join(cmd)}\n{out}")
    return out


def build(verbose: bool = False, debug: bool = False) -> str:
    bdir = os.path.join(BUILD, "debug") if debug else BUILD
    lib = LIB_DEBUG if debug else LIB
    flags = FLAGS + (["-DGPTQ_DEBUG"] if debug else [])
    os.makedirs(bdir, exist_ok=True)
    objs = [os.path.join(bdir, s.replace(".hip", ".o")) for s in SOURCES]
    cmds = [[HIPCC, *flags, "-c", os.path.join(CSRC, s), "-o", o] for s, o in zip(SOURCES, objs)]
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(len(cmds), os.cpu_count() or 4)) as ex:
        for out in ex.map(_run, cmds):
            if verbose and out.strip():
                print(out)
    tmp = lib + ".tmp"
    _run([HIPCC, "-shared", f"--offload-arch={ARCH}", "-o", tmp, *objs])
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, debug="--debug" in sys.argv))
