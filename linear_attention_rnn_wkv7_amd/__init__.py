"""MI355X-native WKV7 (RWKV-7) recurrence: forward scan and reverse scan.

The compute lives in libwkv7.so (hand-written HIP for gfx950 behind a C ABI,
include/wkv7.h; the gated delta rule and the norms around it include/gdr.h,
include/residual_norm.h; softmax attention include/attention.h); ``api`` is a thin torch binding of it.  Importing the
package does not load the library; the first call does, and raises if it
has not been built.
"""
__all__ = ["wkv7_forward", "wkv7_backward", "wkv7_checkpoint_bytes",
           "wkv7_backward_workspace_bytes",
           "gdr_forward", "gdr_backward", "gdr_decode", "gdr_checkpoint_bytes",
           "gdr_forward_workspace_bytes", "gdr_backward_workspace_bytes",
           "gdr_epilogue_forward", "gdr_epilogue_backward", "gdr_epilogue_workspace_bytes",
           "residual_norm_forward", "residual_norm_backward", "residual_norm_workspace_bytes",
           "attn_forward", "attn_backward", "attn_record_bytes", "attn_backward_workspace_bytes",
           "attn_decode", "attn_decode_workspace_bytes", "kv_write", "kv_read",
           "qk_norm_forward", "qk_norm_backward", "qk_norm_workspace_bytes"]


def __getattr__(name):
    if name in __all__:
        from . import api
        return getattr(api, name)
    raise AttributeError(name)
