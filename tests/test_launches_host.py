"""The grids of the rotation, the cache and attention over it at the largest accepted shapes, from a program whose own
hipLaunchKernel writes them down instead of launching (tests/sanitize/abi_launch_driver.cpp)."""
import os

import pytest

from tests.test_sanitizers import ROOT, SAN, _run


@pytest.mark.skipif(not os.path.exists("/opt/rocm/bin/hipcc"), reason="hipcc not installed")
def test_no_launch_passes_the_limits_of_a_grid(tmp_path):
    from bit_ternary_weight_bitlinear_amd import build as hip_build
    objdir = os.path.join(ROOT, "bit_ternary_weight_bitlinear_amd", "_build")
    objs = [os.path.join(objdir, s.replace(".hip", ".o")) for s in hip_build.SOURCES]
    if not all(os.path.exists(o) for o in objs):
        hip_build.build()
    drv, exe = str(tmp_path / "driver.o"), str(tmp_path / "driver")
    _run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__=1", "-I/opt/rocm/include", "-c", os.path.join(SAN, "abi_launch_driver.cpp"), "-o", drv], ROOT)
    _run(["/opt/rocm/bin/hipcc", "--offload-arch=gfx950", drv, *objs, "-o", exe], ROOT)
    assert "abi launch driver: ok" in _run([exe], ROOT).stdout
