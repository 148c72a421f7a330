"""Build the CUDA library libsage.so, and the extension module that hands torch
tensors to its serving calls, in-tree for sm_100a (B200).

    python -m action_diffusion_transformers_b200.build [--verbose]

nvcc compiles csrc/sage_api.cu (quantized attention, projections) and
csrc/serve_api.cu (rotary positions, KV cache, prompt and single-token
attention), each with the kernel headers it includes, side by side and links
them into a shared library with the CUDA runtime linked statically, so the .so
loads on a machine without a GPU (for the symbol checks) and on the B200 machine
alongside torch.  g++ compiles csrc/serve_ext.cpp against the installed torch's
headers into _serve_ext.so, which is linked to libsage.so beside it.
"""
from __future__ import annotations

import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libsage.so")
EXT = os.path.join(PKG, "_serve_ext.so")
EXT_SOURCE = os.path.join(CSRC, "serve_ext.cpp")
SOURCES = [os.path.join(CSRC, "sage_api.cu"), os.path.join(CSRC, "serve_api.cu")]


def deps() -> list:
    """Every file the library is built from: all sources and headers under
    csrc/ and include/ (so an edit to any of them triggers a rebuild)."""
    out = []
    for d in (CSRC, INCLUDE):
        for name in sorted(os.listdir(d)):
            if name.endswith((".cu", ".cuh", ".h", ".cpp")):
                out.append(os.path.join(d, name))
    return out


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def built_for() -> str:
    """What the extension module depends on besides its sources: the torch and the
    Python whose interfaces it was compiled against.  The module carries this text."""
    return f"torch {importlib.metadata.version('torch')}, {sysconfig.get_config_var('SOABI')}"


def ext_command(out: str) -> list:
    """g++ command of the extension module.  It leaves the torch libraries to be
    found where `import torch` has loaded them, and libsage.so beside itself."""
    import torch
    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), INCLUDE]
    return (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", f'-DSAGE_BUILT_FOR="{built_for()}"']
            + [f for d in inc for f in ("-isystem", d)] + [EXT_SOURCE, "-o", out, "-L", os.path.join(root, "lib")]
            + ["-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-L", PKG, "-l:libsage.so", "-Wl,-rpath,$ORIGIN"])


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(EXT):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(EXT))
    with open(EXT, "rb") as f:
        if built_for().encode() + b"\0" not in f.read():
            return False
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
    cmd = ext_command(EXT + ".tmp")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    os.replace(EXT + ".tmp", EXT)
    return LIB


if __name__ == "__main__":
    build(verbose="--verbose" in sys.argv, force=True)
    print(LIB)
