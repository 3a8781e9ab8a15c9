"""Build libconv3d.so (the CUDA library) in-tree with nvcc for sm_100a.

The translation units are compiled side by side into build/ (one object each,
recompiled when it or a header is newer) and linked; then the native Python
binding of the channel-wise operators, _channel.so, against torch's headers
(again when torch or Python is another one than it was built for).
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(ROOT, "build")
LIB = os.path.join(PKG, "libconv3d.so")
BINDING = os.path.join(PKG, "_channel.so")
BUILT_FOR = os.path.join(OBJ, "_channel.built_for")
SOURCES = [os.path.join(CSRC, f) for f in ("conv3d_api.cu", "groupnorm.cu", "channel_ops.cu", "linear.cu")]
# the headers that each unit includes (besides the public one)
HEADERS = {
    "conv3d_api.cu": ("conv3d_kernel.cuh", "wgrad_kernel.cuh", "pipeline.cuh", "ptx.cuh", "internal.h"),
    "groupnorm.cu": (),
    "channel_ops.cu": ("act8.cuh", "ptx.cuh", "internal.h"),
    "linear.cu": ("linear_kernel.cuh", "linear_wgrad.cuh", "act8.cuh", "pipeline.cuh", "ptx.cuh", "internal.h"),
}
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _deps(src: str) -> list[str]:
    own = [os.path.join(CSRC, h) for h in HEADERS[os.path.basename(src)]]
    return [src, os.path.join(ROOT, "include", "conv3d.h"), *own]


def _newer(deps: list[str], than: str) -> bool:
    return not os.path.exists(than) or any(os.path.getmtime(d) > os.path.getmtime(than) for d in deps)


def binding_command() -> list[str]:
    import sysconfig
    import torch
    root = os.path.dirname(torch.__file__)
    includes = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include"),
                sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++20", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *(a for i in includes for a in ("-isystem", i)), "-I", os.path.join(ROOT, "include"),
            "-o", BINDING, os.path.join(CSRC, "binding.cpp"),
            "-L", os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python",
            "-L", PKG, "-l:libconv3d.so", "-Wl,-rpath,$ORIGIN"]


def binding_target() -> str:
    """What the binding is built for: it fits no other torch or Python."""
    from importlib.metadata import version
    return f"torch {version('torch')}, Python {sys.version.split()[0]}\n"


def binding_stale() -> bool:
    deps = [os.path.join(CSRC, "binding.cpp"), os.path.join(ROOT, "include", "conv3d.h")]
    if _newer(deps, BINDING) or not os.path.exists(BUILT_FOR):
        return True
    with open(BUILT_FOR) as f:
        return f.read() != binding_target()


def build(force: bool = False, verbose: bool = False) -> str:
    if force or _newer([d for s in SOURCES for d in _deps(s)], LIB):
        os.makedirs(OBJ, exist_ok=True)
        extra = ["-Xptxas", "-v"] if verbose else []
        running, objects = [], []
        for src in SOURCES:
            obj = os.path.join(OBJ, os.path.basename(src) + ".o")
            objects.append(obj)
            if force or _newer(_deps(src), obj):
                cmd = ["nvcc", *FLAGS, *extra, "-c", "-o", obj, src]
                running.append((cmd, subprocess.Popen(cmd)))
        failed = [cmd for cmd, p in running if p.wait() != 0]
        if failed:
            raise subprocess.CalledProcessError(1, failed[0])
        subprocess.run(["nvcc", "-gencode", "arch=compute_100a,code=sm_100a", "--shared", "-o", LIB, *objects],
                       check=True)
    if force or binding_stale():
        subprocess.run(binding_command(), check=True)
        os.makedirs(OBJ, exist_ok=True)
        with open(BUILT_FOR, "w") as f:
            f.write(binding_target())
    return LIB


if __name__ == "__main__":
    build(force=True, verbose="-v" in sys.argv)
