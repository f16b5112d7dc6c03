"""Build libtilegemm.so (the HIP kernels and the C ABI) for gfx950, in-tree.

Every HIP source is compiled with hipcc for gfx950 only; packed fp32 ALU ops are
disabled (-packed-fp32-ops) and the objects are linked into one shared library
next to this file.  Run ``python -m tiled_dense_gemm_07_amd.build``.
"""

from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libtilegemm.so")
SOURCES = ["tg_api.hip", "tg_gemm_f32.hip", "tg_gemm_f16.hip", "tg_gemm_bf16.hip",
           "tg_dequant_w4.hip", "tg_gemm_mx.hip", "tg_gemm_sp24.hip", "tg_i8.hip", "tg_norm.hip"]
ARCH = "gfx950"
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = ["--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC", "-Wall",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def build(verbose: bool = False) -> str:
    from . import configgen

    configgen.write_all()  # generated configurations (no-op when unchanged)
    return _build_lib(SOURCES + configgen.generated_sources(), LIB, verbose)


def _build_lib(sources, lib_path: str, verbose: bool) -> str:
    os.makedirs(BUILD, exist_ok=True)
    jobs = max(1, min(len(sources), len(os.sched_getaffinity(0))))
    pending = list(sources)
    running = []
    done = []
    objs = [os.path.join(BUILD, src.replace(".hip", ".o")) for src in sources]
    # largest translation units first, at most `jobs` compiles at a time
    pending.sort(key=lambda s: -os.path.getsize(os.path.join(CSRC, s)))
    while pending or running:
        while pending and len(running) < jobs:
            src = pending.pop(0)
            cmd = [HIPCC] + FLAGS + ["-I", os.path.join(HERE, "..", "include"), "-c",
                                     os.path.join(CSRC, src), "-o",
                                     os.path.join(BUILD, src.replace(".hip", ".o"))]
            running.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                                  stderr=subprocess.STDOUT)))
        src, p = running.pop(0)
        out, _ = p.communicate()
        done.append((src, p, out))
    failed = []
    for src, p, out in done:
        text = "\n".join(l for l in out.decode(errors="replace").splitlines()
                         if "not a recognized feature" not in l)
        if verbose and text.strip():
            print(text)
        if p.returncode != 0:
            failed.append((src, text))
    if failed:
        for src, text in failed:
            sys.stderr.write("---- %s ----\n%s\n" % (src, text))
        raise RuntimeError("hipcc failed for: " + ", ".join(s for s, _ in failed))
    tmp = lib_path + ".tmp%d" % os.getpid()
    subprocess.run([HIPCC, "--offload-arch=" + ARCH, "-shared", "-fPIC", "-o", tmp] + objs,
                   check=True)
    os.replace(tmp, lib_path)
    return lib_path


if __name__ == "__main__":
    print(build(verbose=True))
