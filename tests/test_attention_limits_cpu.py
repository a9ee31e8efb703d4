"""Limits of softmax attention's calls that are refused, without a GPU."""
import ctypes

import pytest

from linear_attention_rnn_wkv7_amd import _lib
from test_attention_cpu import FAKE, INVALID, WORKSPACE, attn_shape, decode_shape


@pytest.mark.parametrize("scale, ok", [(2.0 ** 127, True), (2.0 ** 127 * (1 + 2.0 ** -23), False), (3.4028234e38, False), (2.0 ** -126, True)])
def test_largest_scale(scale, ok):
    """scale log2 e has to be finite in fp32: with an infinity there, a score of 0 would
    have NaN for a weight."""
    L = _lib.lib()
    r = ctypes.byref(attn_shape(scale=scale))
    assert (L.attn_backward_workspace_bytes(r) > 0) == ok and (L.attn_record_bytes(r) > 0) == ok
    # (no workspace: refused before anything is enqueued)
    assert L.attn_backward(r, *[FAKE] * 3, None, FAKE, FAKE, None, *[FAKE] * 4, None, 0, None) == (WORKSPACE if ok else INVALID)
    if not ok:
        assert L.attn_forward(r, *[FAKE] * 3, None, FAKE, None, None, None) == INVALID
    r = ctypes.byref(decode_shape(scale=scale))
    assert (L.attn_decode_workspace_bytes(r) > 0) == ok
    assert L.attn_decode(r, *[FAKE] * 3, None, None, *[FAKE] * 3, None, 0, None) == (WORKSPACE if ok else INVALID)
