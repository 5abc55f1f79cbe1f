"""The host side of the attention and cache calls (argument checks, workspace and launch arithmetic) under
AddressSanitizer and UndefinedBehaviorSanitizer, host code only, in an executable of its own."""
import os

import pytest

from tests.test_sanitizers import ROOT, SAN, _run


@pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="hipcc not installed")
def test_attention_host_code_under_asan_ubsan(tmp_path):
    from concurrent.futures import ThreadPoolExecutor

    from bit_ternary_weight_bitlinear_amd import build as hip_build
    hipcc = "/opt/rocm/bin/hipcc"
    csrc = os.path.join(ROOT, "bit_ternary_weight_bitlinear_amd", "csrc")
    objdir = os.path.join(ROOT, "bit_ternary_weight_bitlinear_amd", "_build")
    checked = ["api.hip", "attention.hip", "attention_cached.hip", "cache.hip"]
    others = [os.path.join(objdir, s.replace(".hip", ".o")) for s in hip_build.SOURCES if s not in checked]
    if not all(os.path.exists(o) for o in others):
        hip_build.build()
    san = ["-fsanitize=address", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer"]
    host_san = [a for f in san for a in ("-Xarch_host", f)]

    def compile_one(src):
        obj = str(tmp_path / src.replace(".hip", ".o"))
        # device code as small as it gets: none of it is run
        _run([hipcc, *hip_build.FLAGS, *host_san, "-Xarch_device", "-O1", "-g", "-c", os.path.join(csrc, src), "-o", obj], ROOT)
        return obj

    with ThreadPoolExecutor(len(checked)) as ex:
        objs = list(ex.map(compile_one, checked))
    drv = str(tmp_path / "driver.o")
    _run(["g++", "-std=c++17", "-g", *san, "-D__HIP_PLATFORM_AMD__=1", "-I/opt/rocm/include", "-c", os.path.join(SAN, "abi_attention_driver.cpp"),
          "-o", drv], ROOT)
    exe = str(tmp_path / "driver")
    _run([hipcc, "--offload-arch=gfx950", *host_san, drv, *objs, *others, "-o", exe], ROOT)
    r = _run([exe], ROOT)
    assert "abi attention driver: ok" in r.stdout
