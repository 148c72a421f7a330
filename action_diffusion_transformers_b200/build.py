"""Build the CUDA library libsage.so in-tree for sm_100a (B200).

    python -m action_diffusion_transformers_b200.build [--verbose]

nvcc compiles csrc/sage_api.cu (quantized attention, projections) and
csrc/serve_api.cu (rotary positions, KV cache, prompt and single-token
attention), each with the kernel headers it includes, side by side and links
them into a shared library with the CUDA runtime linked statically, so the .so
loads on a machine without a GPU (for the symbol checks) and on the B200 machine
alongside torch.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libsage.so")
SOURCES = [os.path.join(CSRC, "sage_api.cu"), os.path.join(CSRC, "serve_api.cu")]


def deps() -> list:
    """Every file the library is built from: all sources and headers under
    csrc/ and include/ (so an edit to any of them triggers a rebuild)."""
    out = []
    for d in (CSRC, INCLUDE):
        for name in sorted(os.listdir(d)):
            if name.endswith((".cu", ".cuh", ".h")):
                out.append(os.path.join(d, name))
    return out


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in deps())


def build(verbose: bool = False, force: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    flags = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3", "-std=c++17",
             "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC]
    if verbose:
        flags.insert(0, "-Xptxas=-v")
    with tempfile.TemporaryDirectory() as tmp:
        objs = [os.path.join(tmp, os.path.basename(src) + ".o") for src in SOURCES]
        cmds = [[nvcc()] + flags + ["-c", "-o", obj, src] for src, obj in zip(SOURCES, objs)]
        runs = [subprocess.Popen(c, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True) for c in cmds]
        for cmd, (out, rc) in zip(cmds, [(r.communicate()[0], r.returncode) for r in runs]):
            if rc != 0:
                raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + out)
            if verbose:
                sys.stdout.write(out)
        cmd = [nvcc()] + flags + ["-shared", "-o", LIB + ".tmp"] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(verbose="--verbose" in sys.argv, force=True)
    print(LIB)
