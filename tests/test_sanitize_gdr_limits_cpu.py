"""The size limits of the gated delta rule and the norms under
AddressSanitizer and UndefinedBehaviorSanitizer (CPU only), with the kernel
launchers replaced by recording stubs."""
import os
import shutil

import pytest

from test_sanitize_cpu import HERE, ROOT, SAN, _check, _run


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the HIP headers not available")
def test_gdr_limits_under_sanitizers(tmp_path):
    exe = str(tmp_path / "gdr_limits_driver")
    csrc = os.path.join(ROOT, "linear_attention_rnn_wkv7_amd", "csrc")
    rc, out = _run(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I", os.path.join(ROOT, "include"), "-I", csrc, "-o", exe,
                    os.path.join(HERE, "gdr_limits_driver.cpp"), os.path.join(csrc, "gdr_abi.cpp")])
    assert rc == 0, out
    _check(exe)
