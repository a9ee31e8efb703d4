"""The size limits of the gated delta rule and the norms under
AddressSanitizer and UndefinedBehaviorSanitizer (CPU only), with the kernel
launchers replaced by recording stubs."""
import ctypes
import os
import shutil

import pytest

from linear_attention_rnn_wkv7_amd import _lib
from test_sanitize_cpu import HERE, ROOT, SAN, _check, _run

UNSUPPORTED = _lib.WKV7_ERR_UNSUPPORTED


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


def test_rule_at_its_limits():
    """2^22 chunks of one head are within the limit; a shape whose scan would
    launch 2^32 threads is refused before anything is launched."""
    L = _lib.lib()

    def shape(B, T, H, V, dtype=1):
        return ctypes.byref(_lib.GdrShape(B, T, H, H, 64, V, 0, dtype, 0, 0.125))

    assert L.gdr_checkpoint_bytes(shape(64, 64 * 65536, 1, 64)) == 2 ** 22 * (64 * 64 + 64 * 64) * 4
    big = shape(65535, 1, 64, 256)
    fake = 0x10000
    assert L.gdr_forward_workspace_bytes(big) == 0 and L.gdr_backward_workspace_bytes(big, 1) == 0
    for y, sT in ((fake, None), (fake, fake)):
        assert L.gdr_forward(big, *[fake] * 5, None, None, y, sT, None, fake, 1 << 45, None) == UNSUPPORTED
    assert L.gdr_backward(big, *[fake] * 5, None, None, fake, None, fake, *[fake] * 6, fake, 1 << 45, None) == UNSUPPORTED
    assert L.gdr_checkpoint_bytes(shape(65535, 1, 64, 128)) > 0
