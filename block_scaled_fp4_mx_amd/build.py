"""Build libfp4.so (gfx950) in-tree with hipcc.

Each translation unit under csrc/ is compiled to an object in parallel, then
linked into block_scaled_fp4_mx_amd/libfp4.so.  csrc/binding.cpp, host code that
sees torch's tensors, becomes the extension module _binding.so beside it.  The
peak-rate microbenchmarks (probes/peak.hip, not part of the library) build into
probes/libfp4_peak.so.  Every build recompiles.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libfp4.so")
BINDING_OUT = os.path.join(HERE, "_binding.so")
BUILD = os.path.join(HERE, "_build")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

SOURCES = ["api.cpp", "quant.hip", "gemm.hip", "moe.hip", "qk_norm.hip", "rope_append.hip", "kv_pages.hip",
           "attn_tree.hip", "attn_shared.hip", "attn_blocks.hip", "kv_select.hip", "attn_prompt.hip"]
PROBES = os.path.join(HERE, "probes")
PROBE_OUT = os.path.join(PROBES, "libfp4_peak.so")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Wall",
    # packed fp32 VALU ops stay off (scalar fp32 code only)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(HERE, "..", "include"),
]


def _run(what: str, cmd: list[str]) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return r.stderr


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    err = _run(f"hipcc for {src}", [HIPCC, "-x", "hip", *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj])
    if err.strip():
        sys.stderr.write(err)
    return obj


def _compile_binding() -> str:
    obj = os.path.join(BUILD, "binding.o")
    torch = os.path.join(os.path.dirname(importlib.util.find_spec("torch").origin), "include")
    _run("hipcc for binding.cpp",
         [HIPCC, "-x", "c++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
          "-I", os.path.join(HERE, "..", "include"), "-I", sysconfig.get_paths()["include"], "-isystem", torch,
          "-isystem", os.path.join(torch, "torch", "csrc", "api", "include"), "-isystem", "/opt/rocm/include",
          "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj])
    return obj


def _link_binding(obj: str) -> None:
    """Against libfp4.so beside it and torch's libraries, which importing torch has loaded."""
    tmp = BINDING_OUT + ".tmp"
    libs = os.path.join(os.path.dirname(importlib.util.find_spec("torch").origin), "lib")
    _run("link of _binding.so",
         [HIPCC, "-shared", "-fPIC", "-o", tmp, obj, "-L", HERE, "-l:" + os.path.basename(OUT), "-Wl,-rpath,$ORIGIN",
          "-L", libs, "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_python"])
    os.replace(tmp, BINDING_OUT)


def _build_probes() -> None:
    tmp = PROBE_OUT + ".tmp"
    _run("hipcc for probes/peak.hip", [HIPCC, "-x", "hip", *FLAGS, "-shared", os.path.join(PROBES, "peak.hip"), "-o", tmp])
    os.replace(tmp, PROBE_OUT)


def build(verbose: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, len(SOURCES) + 2)) as ex:
        probes = ex.submit(_build_probes)
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(_compile, SOURCES))
        probes.result()
        binding_obj = binding.result()
    tmp = OUT + ".tmp"
    _run("link", [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs])
    os.replace(tmp, OUT)
    _link_binding(binding_obj)
    if verbose:
        print(f"built {OUT}, {BINDING_OUT} and {PROBE_OUT}")
    return OUT


if __name__ == "__main__":
    build()
