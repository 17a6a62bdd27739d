"""Build libbmmc.so (HIP kernels for gfx950 + host planner + C ABI) in-tree.

    python -m bmmc_affine_index_amd.build

compiles every source under csrc/ with hipcc into _build/ and links
bmmc_affine_index_amd/libbmmc.so, and the binding of the calls on torch's
tensors, bmmc_affine_index_amd/_calls.so.  hipcc cross-compiles for gfx950
without a GPU.  Every HIP source is built with packed-FP32 instructions disabled.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libbmmc.so")
CALLS = os.path.join(PKG, "_calls.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

COMMON = ["-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-function",
          "-I" + os.path.join(ROOT, "include")]
HIP_FLAGS = ["--offload-arch=" + ARCH, "-Xclang", "-target-feature", "-Xclang",
             "-packed-fp32-ops", "-munsafe-fp-atomics"]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cpp")) + glob.glob(os.path.join(CSRC, "*.hip")) +
                  glob.glob(os.path.join(CSRC, "kernels", "*.hip")) +
                  glob.glob(os.path.join(CSRC, "tokens", "*.cpp")) +
                  glob.glob(os.path.join(CSRC, "tokens", "*.hip")))


def binding_sources():
    return sorted(glob.glob(os.path.join(CSRC, "binding", "*.cpp")))


def _torch_dir() -> str:
    """torch's folder, found without importing it."""
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def _compile(src: str) -> str:
    rel = os.path.relpath(src, CSRC).replace(os.sep, "_")
    obj = os.path.join(BUILD, rel + ".o")
    cmd = [HIPCC] + COMMON
    if src in binding_sources():
        cmd += ["-DUSE_ROCM", "-isystem", os.path.join(_torch_dir(), "include"),
                "-isystem", sysconfig.get_paths()["include"]]
    if src.endswith(".hip"):
        cmd += HIP_FLAGS + ["-x", "hip"]
    else:
        cmd += ["-x", "c++", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include"]
    cmd += ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("compile failed: %s\n%s\n%s" % (" ".join(cmd), r.stdout, r.stderr))
    return obj


def _link(objs, out: str, more) -> None:
    tmp = out + ".tmp"
    cmd = [HIPCC, "-shared", "-fPIC"] + objs + more + ["-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed: %s\n%s\n%s" % (" ".join(cmd), r.stdout, r.stderr))
    os.replace(tmp, out)


def build(jobs: int = 8) -> str:
    """Compile all sources and link libbmmc.so and _calls.so; returns the
    library's path."""
    os.makedirs(BUILD, exist_ok=True)
    srcs, binding = sources(), binding_sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(jobs, len(srcs) + len(binding)))) as ex:
        objs = list(ex.map(_compile, binding + srcs))
    _link(objs[len(binding):], LIB, ["--offload-arch=" + ARCH])
    # torch's libraries are loaded before the binding is, by `import torch`
    _link(objs[:len(binding)], CALLS,
          ["-no-hip-rt", "-L" + os.path.join(_torch_dir(), "lib"), "-lc10", "-lc10_hip",
           "-ltorch_cpu", "-ltorch_python"])
    return LIB


if __name__ == "__main__":
    print(build(int(sys.argv[1]) if len(sys.argv) > 1 else 8))
