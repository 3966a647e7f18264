"""AddressSanitizer + UndefinedBehaviorSanitizer build of the host code of the
operators around the forward (kda_grad_api.cpp, kda_ops_api.cpp), on the CPU, driven
over random and extreme descriptors (tests/sanitize/ops_driver.cpp)."""
import os

import pytest

from test_sanitize import ENV, ROOT, SAN, SAN_FLAGS, need, run


def test_ops_host_code_under_sanitizers(tmp_path):
    need("g++")
    if not os.path.isdir("/opt/rocm/include/hip"):
        pytest.skip("HIP headers not installed")
    exe = str(tmp_path / "ops_driver")
    src = os.path.join(ROOT, "gated_delta_rule_63_amd", "csrc")
    cmd = ["g++", "-std=c++17", *SAN_FLAGS, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
           *(os.path.join(src, f) for f in ("kda_grad_api.cpp", "kda_ops_api.cpp", "kda_api.cpp")),
           os.path.join(SAN, "launch_stubs.cpp"), os.path.join(SAN, "ops_driver.cpp"),
           "-L/opt/rocm/lib", "-Wl,-rpath,/opt/rocm/lib", "-lamdhip64", "-o", exe]
    rc, out = run(cmd)
    assert rc == 0, out
    # HIP_VISIBLE_DEVICES="" keeps the driver off any GPU: only host code runs
    rc, out = run([exe], env=dict(ENV, HIP_VISIBLE_DEVICES=""), timeout=120)
    assert rc == 0 and "runtime error" not in out and "AddressSanitizer" not in out, out
    assert "all expectations met" in out
