"""Compile the gfx950 HIP sources into bit_ternary_weight_bitlinear_amd/libbitlinear.so
(the product library) and libbitlinear_bench.so (the benchmark's plain read
kernels, loaded by bench.py only), and the host-only module _binding.so, which
marshals torch tensors to the library's attention calls. The library needs hipcc
alone and is linked first; where torch is not installed the module is left out.

Flags: correctly rounded fp32 division, no FMA contraction, no fast-math, no
denormal flushing (the quantizers decide integers in fp32 and must match the
definition bit for bit), and packed-fp32 instructions disabled.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libbitlinear.so")
BENCH_LIB = os.path.join(HERE, "libbitlinear_bench.so")
SOURCES = ["api.hip", "pack.hip", "act_quant.hip", "gemv.hip", "bgemv.hip", "gemm.hip", "skinny.hip",
           "sparse_down.hip", "bmma.hip", "attention.hip", "attention_cached.hip", "cache.hip"]
BENCH_SOURCES = ["bench_read.hip"]
BINDING = os.path.join(HERE, "_binding.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-ffp-contract=off", "-fno-fast-math",
    "-fhip-fp32-correctly-rounded-divide-sqrt", "-fno-gpu-flush-denormals-to-zero",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]
# Where LDS lets one workgroup of four waves onto a CU, a wave may have more than 256
# registers and the compiler puts matrix results into the accumulation half of them,
# which vector instructions reach by copies only: this keeps them in the other.
EXTRA_FLAGS = {"attention.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]}


def build_binding(verbose: bool = False) -> str | None:
    """The CPython module of the attention calls (csrc/binding.cpp, host code only); None without torch,
    whose tensors it takes."""
    try:
        import torch
    except ImportError as e:
        print(f"{BINDING} is not built ({e}); the C library does not need it", file=sys.stderr)
        return None
    base = os.path.dirname(torch.__file__)
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f"-I{base}/include", f"-I{base}/include/torch/csrc/api/include", "-I/opt/rocm/include",
           f"-I{sysconfig.get_paths()['include']}", os.path.join(CSRC, "binding.cpp"), "-o", BINDING + ".tmp",
           f"-L{base}/lib", "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_python", "-ldl"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{r.stderr}")
    os.replace(BINDING + ".tmp", BINDING)
    return BINDING


def build(verbose: bool = False, out_dir: str | None = None) -> str:
    out_dir = out_dir or os.path.join(HERE, "_build")
    os.makedirs(out_dir, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(out_dir, src.replace(".hip", ".o"))
        cmd = [HIPCC, *FLAGS, *EXTRA_FLAGS.get(src, []), "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
        if verbose and r.stderr.strip():
            print(r.stderr, flush=True)
        return obj

    all_src = SOURCES + BENCH_SOURCES
    with ThreadPoolExecutor(max_workers=min(len(all_src), os.cpu_count() or 1)) as ex:
        binding = ex.submit(build_binding, verbose)
        objs = dict(zip(all_src, ex.map(compile_one, all_src)))
    for lib, srcs in ((LIB, SOURCES), (BENCH_LIB, BENCH_SOURCES)):
        cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *[objs[s] for s in srcs], "-o", lib + ".tmp"]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        os.replace(lib + ".tmp", lib)
    binding.result()  # raises what the module's compiler reported
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
