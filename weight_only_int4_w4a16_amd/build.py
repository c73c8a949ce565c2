"""Build libw4a16.so (hipcc, for gfx950) and _binding.so (the C++ part of the Python binding) in-tree.

    python -m weight_only_int4_w4a16_amd.build [--jobs N] [extra hipcc flags]

Every HIP source is compiled with the packed-FP32 feature switched off
(-Xclang -target-feature -Xclang -packed-fp32-ops): ordinary float code only.
"""
from __future__ import annotations

import os
import shlex
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libw4a16.so")
SOURCES = ["kernels.hip", "kernels3.hip", "quantize.hip", "stream_probe.hip", "api.hip", "plan.cpp",
           "page_tables.hip", "kv_write.hip", "paged_attention.hip", "linear_attention.hip",
           "delta_rule.hip", "quantized_kv.hip", "quantized_attention.hip", "api_mixers.hip"]
BINDING = os.path.join(PKG, "_binding.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

COMMON = ["-O3", "-std=c++17", "-fPIC", "--offload-arch=gfx950",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-fhip-fp32-correctly-rounded-divide-sqrt",
          "-Wall", "-Wno-unused-function", "-I", INCLUDE, "-I", CSRC]


def build_binding(out: str = BINDING) -> str:
    """The Python module over torch's C++ API (csrc/binding.cpp); host code only."""
    import torch
    from torch.utils import cpp_extension
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = out + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-D__HIP_PLATFORM_AMD__=1",
           "-I", INCLUDE, *(x for p in cpp_extension.include_paths() for x in ("-isystem", p)),
           "-isystem", os.path.join(os.path.dirname(os.path.dirname(HIPCC)), "include"),
           "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, "binding.cpp"),
           "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip", f"-Wl,-rpath,{lib}", "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{shlex.join(cmd)}\n{r.stderr}")
    os.replace(tmp, out)
    return out


def build(out: str = LIB, extra=(), build_dir: str | None = None, jobs: int = 4) -> str:
    build_dir = build_dir or os.path.join(PKG, "_build")
    os.makedirs(build_dir, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(build_dir, src + ".o")
        lang = ["-x", "hip"] if src.endswith(".hip") else ["-x", "c++"]
        cmd = [HIPCC, *COMMON, *extra, *lang, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"hipcc failed for {src}:\n{shlex.join(cmd)}\n{r.stderr}")
        return obj

    with ThreadPoolExecutor(max_workers=max(1, jobs)) as ex:
        binding = ex.submit(build_binding)
        objs = list(ex.map(compile_one, SOURCES))
        binding.result()
    tmp = out + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{shlex.join(cmd)}\n{r.stderr}")
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    args = sys.argv[1:]
    jobs = 4
    if args[:1] == ["--jobs"]:
        jobs, args = int(args[1]), args[2:]
    print(build(extra=args, jobs=jobs))
