"""The order of attention's workgroups over rows, heads and tiles (CPU only): a
mapping that takes each of them once."""
import os
import shutil

import pytest

from test_sanitize_cpu import HERE, ROOT, SAN, _check, _run


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir("/opt/rocm/include"),
                    reason="g++ or the HIP headers not available")
def test_every_tile_is_one_workgroups(tmp_path):
    exe = str(tmp_path / "attn_tiles_driver")
    csrc = os.path.join(ROOT, "linear_attention_rnn_wkv7_amd", "csrc")
    rc, out = _run(["g++", "-std=c++17", *SAN, "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I", os.path.join(ROOT, "include"), "-I", csrc, "-o", exe,
                    os.path.join(HERE, "attn_tiles_driver.cpp")])
    assert rc == 0, out
    _check(exe)
