"""Sizes and messages of the torch binding of the gated delta rule and the
norms, without a GPU."""
import ctypes

import torch

import linear_attention_rnn_wkv7_amd as pkg
from linear_attention_rnn_wkv7_amd import _lib


def test_norm_workspace_sizes():
    """What `workspace=` of the norms' backwards has to hold."""
    L = _lib.lib()
    for rows, H, N, per_head, dt in ((3, 4, 64, False, torch.float32), (70000, 32, 128, True, torch.bfloat16), (0, 3, 64, True, torch.float32)):
        sh = _lib.GdrEpilogueShape(rows, H, N, H if per_head else 1, int(dt == torch.bfloat16), 0, 1e-6)
        want = L.gdr_epilogue_workspace_bytes(ctypes.byref(sh))
        assert pkg.gdr_epilogue_workspace_bytes(rows, H, N, H if per_head else 1, dt) == want
        assert (want > 0) == (rows > 0)
    for rows, D, dt in ((3, 100, torch.float32), (100000, 2047, torch.bfloat16), (0, 5, torch.bfloat16)):
        sh = _lib.ResidualNormShape(rows, D, int(dt == torch.bfloat16), 0, 1e-6)
        want = L.residual_norm_workspace_bytes(ctypes.byref(sh))
        assert pkg.residual_norm_workspace_bytes(rows, D, dt) == want
        assert (want > 0) == (rows > 0)
    assert "gdr_epilogue_workspace_bytes" in pkg.__all__ and "residual_norm_workspace_bytes" in pkg.__all__


def test_sizes_of_a_rule_without_a_key():
    """K = 0 is refused like other sizes, though the default scale is K ** -0.5."""
    assert pkg.gdr_checkpoint_bytes(1, 5, 1, 1, 0, 16) == 0
    assert pkg.gdr_forward_workspace_bytes(1, 5, 1, 1, 0, 16) == 0
    assert pkg.gdr_backward_workspace_bytes(1, 5, 1, 1, 0, 16) == 0


def test_unsupported_says_what_of():
    """The text for a size that a call does not take is not only about wkv7's
    head sizes."""
    text = _lib.status_text(_lib.WKV7_ERR_UNSUPPORTED)
    assert "a size that the call does not take" in text and "gdr.h" in text and "residual_norm.h" in text
