"""Build libssd.so (the gfx950 HIP kernels and the C ABI) and _ssd_torch.so (the
host-only calls on torch tensors) in-tree with hipcc.

Every source is compiled for gfx950 only, in parallel, then linked into
state_space_model_amd/libssd.so.  Packed float32 instructions are disabled
(-packed-fp32-ops) for every device compilation.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libssd.so")
BINDING = os.path.join(PKG, "_ssd_torch.so")

SOURCES = ["ssd_api.cpp", "ssd_step.hip", "ssd_state_pass.hip", "ssd_prefill_f32.hip",
           "ssd_prefill_bf16.hip", "ssd_conv.hip", "ssd_backward.hip", "ssd_block_api.cpp",
           "ssd_norm.hip", "ssd_linear_q8.hip", "ssd_conv_backward.hip", "ssd_delta_api.cpp",
           "ssd_delta.hip", "ssd_delta_backward.hip"]
BINDING_SOURCE = "ssd_torch.cpp"
ARCH = "gfx950"


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: libssd.so cannot be built")


def _flags():
    return ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-I", INCLUDE, "-I", CSRC,
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-Wall", "-Wno-unused-function", "-Wno-unused-variable"]


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch not found: _ssd_torch.so cannot be built")
    return spec.submodule_search_locations[0]


def _host_flags():
    torch = _torch_dir()
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(hipcc())))
    return ["-O2", "-std=c++17", "-fPIC", "-D__HIP_PLATFORM_AMD__=1", "-I", INCLUDE,
            "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(torch, "include"),
            "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
            "-isystem", os.path.join(rocm, "include"), "-Wall"]


def _run(what: str, cmd) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    lang = ["-x", "hip"] if src.endswith(".cpp") else []
    flags = _flags()
    if src == BINDING_SOURCE:
        lang, flags = ["-x", "c++"], _host_flags()
    _run("compile", [hipcc()] + lang + flags + ["-c", os.path.join(CSRC, src), "-o", obj])
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    sources = SOURCES + [BINDING_SOURCE]
    jobs = min(len(sources), int(os.environ.get("MAX_JOBS", os.cpu_count() or 4)))
    with cf.ThreadPoolExecutor(max_workers=max(1, jobs)) as ex:
        objs = list(ex.map(_compile, sources))
    tmp = LIB + ".tmp"
    _run("link", [hipcc(), "-shared", "-fPIC", f"--offload-arch={ARCH}", "-o", tmp] + objs[:-1])
    os.replace(tmp, LIB)
    tmp = BINDING + ".tmp"
    _run("link", [hipcc(), "-no-hip-rt", "-shared", "-fPIC", "-o", tmp, objs[-1], "-L", PKG,
                  "-l:libssd.so", "-Wl,-rpath,$ORIGIN", "-L", os.path.join(_torch_dir(), "lib"),
                  "-ltorch_python", "-ltorch_cpu", "-lc10"])
    os.replace(tmp, BINDING)
    if verbose:
        print(LIB)
        print(BINDING)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
