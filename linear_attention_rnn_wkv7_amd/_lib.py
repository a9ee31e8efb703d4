"""ctypes view of libwkv7.so (declarations mirror include/wkv7.h).

WKV7_LIB, when set, names another build of the library to load instead of
the in-tree one (for A/B timing of builds); it must exist.
"""
import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("WKV7_LIB") or os.path.join(PKG, "libwkv7.so")

WKV7_F32, WKV7_BF16 = 0, 1
WKV7_ALGO_AUTO, WKV7_ALGO_SCAN, WKV7_ALGO_CHUNKED = 0, 1, 2
WKV7_OK, WKV7_ERR_INVALID, WKV7_ERR_UNSUPPORTED, WKV7_ERR_WORKSPACE, WKV7_ERR_HIP = 0, -1, -2, -3, -4

# Every function the C header declares, for the symbol-export test.
EXPORTS = ("wkv7_checkpoint_bytes", "wkv7_backward_workspace_bytes", "wkv7_forward",
           "wkv7_backward", "wkv7_epilogue_workspace_bytes", "wkv7_epilogue_forward",
           "wkv7_epilogue_backward", "wkv7_status_string", "wkv7_abi_version",
           "wkv7_fault_status", "wkv7_test_hook", "wkv7_backward_noalloc")
# ... and every function include/rwkv8.h declares
RWKV8_EXPORTS = ("rwkv8_checkpoint_bytes", "rwkv8_backward_workspace_bytes", "rwkv8_forward",
                 "rwkv8_backward")
# ... include/gdr.h and include/residual_norm.h
GDR_EXPORTS = ("gdr_checkpoint_bytes", "gdr_forward_workspace_bytes", "gdr_backward_workspace_bytes",
               "gdr_forward", "gdr_backward", "gdr_decode", "gdr_epilogue_workspace_bytes",
               "gdr_epilogue_forward", "gdr_epilogue_backward")
RESIDUAL_NORM_EXPORTS = ("residual_norm_workspace_bytes", "residual_norm_forward",
                         "residual_norm_backward")
# ... include/attention.h
ATTENTION_EXPORTS = ("attn_record_bytes", "attn_backward_workspace_bytes", "attn_forward", "attn_backward",
                     "qk_norm_workspace_bytes", "qk_norm_forward", "qk_norm_backward", "kv_write", "kv_read",
                     "attn_decode_workspace_bytes", "attn_decode")
WKV7_FAULT_RWKV8_DECAY = 2

WKV7_NOALLOC_SCRATCH_BYTES = 128 << 20

WKV7_FAULT_HELPER_WAIT = 1
WKV7_HOOK_FAULT_INJECT, WKV7_HOOK_FAIL_LAUNCHES = 1, 2


WKV7_FUSED_INPUTS = 1   # wkv7_shape.flags bit


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("H", ctypes.c_int64),
                ("N", ctypes.c_int64), ("dtype", ctypes.c_int32), ("chunk", ctypes.c_int32),
                ("algo", ctypes.c_int32), ("flags", ctypes.c_int32)]


class Rwkv8Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("H", ctypes.c_int64),
                ("Hv", ctypes.c_int64), ("L", ctypes.c_int64), ("E", ctypes.c_int64)]


GDR_NORM_QK = 1   # gdr_shape.flags bit


class GdrShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("Hk", ctypes.c_int64),
                ("Hv", ctypes.c_int64), ("K", ctypes.c_int64), ("V", ctypes.c_int64),
                ("nseq", ctypes.c_int64), ("dtype", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("scale", ctypes.c_float)]


class GdrEpilogueShape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("H", ctypes.c_int64), ("N", ctypes.c_int64),
                ("Hw", ctypes.c_int64), ("dtype", ctypes.c_int32), ("flags", ctypes.c_int32),
                ("eps", ctypes.c_float)]


class ResidualNormShape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("D", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("flags", ctypes.c_int32), ("eps", ctypes.c_float)]


class AttnShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("Hq", ctypes.c_int64),
                ("Hk", ctypes.c_int64), ("D", ctypes.c_int64), ("nseq", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_int32), ("scale", ctypes.c_float)]


QK_NORM_INTERLEAVED = 1   # qk_norm_shape.flags bit


class QkNormShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("Hq", ctypes.c_int64),
                ("Hk", ctypes.c_int64), ("D", ctypes.c_int64), ("R", ctypes.c_int64),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_int32), ("eps", ctypes.c_float)]


KV_CACHE_SAME, KV_CACHE_E4M3 = 0, 1


class KvCacheShape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("T", ctypes.c_int64), ("Hk", ctypes.c_int64),
                ("D", ctypes.c_int64), ("packed", ctypes.c_int64), ("pages", ctypes.c_int64),
                ("page", ctypes.c_int64), ("max_pages", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("dtype", ctypes.c_int32), ("cache_dtype", ctypes.c_int32)]


class AttnDecodeShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("T", ctypes.c_int64), ("Hq", ctypes.c_int64),
                ("Hk", ctypes.c_int64), ("D", ctypes.c_int64), ("pages", ctypes.c_int64),
                ("page", ctypes.c_int64), ("max_pages", ctypes.c_int64), ("q_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int32), ("cache_dtype", ctypes.c_int32), ("scale", ctypes.c_float)]


class Wkv7Error(RuntimeError):
    def __init__(self, func, status, text):
        super().__init__(f"{func} failed: {status} ({text})")
        self.status = status


_LIB = None


def lib():
    """Load libwkv7.so; raise if it has not been built (there is no fallback)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m linear_attention_rnn_wkv7_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
    sp = ctypes.POINTER(Shape)
    L.wkv7_checkpoint_bytes.argtypes = [sp]
    L.wkv7_checkpoint_bytes.restype = sz
    L.wkv7_backward_workspace_bytes.argtypes = [sp, i32]
    L.wkv7_backward_workspace_bytes.restype = sz
    L.wkv7_forward.argtypes = [sp] + [vp] * 10 + [vp]
    L.wkv7_forward.restype = i32
    L.wkv7_backward.argtypes = [sp] + [vp] * 17 + [vp, sz, vp]
    L.wkv7_backward.restype = i32
    L.wkv7_backward_noalloc.argtypes = [sp] + [vp] * 17 + [vp]
    L.wkv7_backward_noalloc.restype = i32
    L.wkv7_epilogue_workspace_bytes.argtypes = [sp]
    L.wkv7_epilogue_workspace_bytes.restype = sz
    L.wkv7_epilogue_forward.argtypes = [sp] + [vp] * 9 + [vp]
    L.wkv7_epilogue_forward.restype = i32
    L.wkv7_epilogue_backward.argtypes = [sp] + [vp] * 17 + [vp, sz, vp]
    L.wkv7_epilogue_backward.restype = i32
    L.wkv7_status_string.argtypes = [i32]
    L.wkv7_status_string.restype = ctypes.c_char_p
    L.wkv7_abi_version.argtypes = []
    L.wkv7_abi_version.restype = i32
    L.wkv7_fault_status.argtypes = [ctypes.POINTER(ctypes.c_uint), i32, vp]
    L.wkv7_fault_status.restype = i32
    L.wkv7_test_hook.argtypes = [i32, ctypes.c_int64]
    L.wkv7_test_hook.restype = i32
    s8 = ctypes.POINTER(Rwkv8Shape)
    L.rwkv8_checkpoint_bytes.argtypes = [s8]
    L.rwkv8_checkpoint_bytes.restype = sz
    L.rwkv8_backward_workspace_bytes.argtypes = [s8, i32]
    L.rwkv8_backward_workspace_bytes.restype = sz
    L.rwkv8_forward.argtypes = [s8] + [vp] * 9 + [vp]
    L.rwkv8_forward.restype = i32
    L.rwkv8_backward.argtypes = [s8] + [vp] * 14 + [vp, sz, vp]
    L.rwkv8_backward.restype = i32
    sg, se, sn = (ctypes.POINTER(x) for x in (GdrShape, GdrEpilogueShape, ResidualNormShape))
    sa, sq, sc, sd = (ctypes.POINTER(x) for x in (AttnShape, QkNormShape, KvCacheShape, AttnDecodeShape))
    i64 = ctypes.c_int64
    for name, args, res in (
            ("gdr_checkpoint_bytes", [sg], sz),
            ("gdr_forward_workspace_bytes", [sg], sz),
            ("gdr_backward_workspace_bytes", [sg, i32], sz),
            ("gdr_forward", [sg] + [vp] * 10 + [vp, sz, vp], i32),
            ("gdr_backward", [sg] + [vp] * 16 + [vp, sz, vp], i32),
            ("gdr_decode", [sg] + [vp] * 6 + [i64, vp, vp, vp], i32),
            ("gdr_epilogue_workspace_bytes", [se], sz),
            ("gdr_epilogue_forward", [se] + [vp] * 4 + [vp], i32),
            ("gdr_epilogue_backward", [se] + [vp] * 7 + [vp, sz, vp], i32),
            ("residual_norm_workspace_bytes", [sn], sz),
            ("residual_norm_forward", [sn] + [vp] * 6 + [vp], i32),
            ("residual_norm_backward", [sn] + [vp] * 10 + [vp, sz, vp], i32),
            ("attn_record_bytes", [sa], sz),
            ("attn_backward_workspace_bytes", [sa], sz),
            ("attn_forward", [sa] + [vp] * 7 + [vp], i32),
            ("attn_backward", [sa] + [vp] * 11 + [vp, sz, vp], i32),
            ("qk_norm_workspace_bytes", [sq], sz),
            ("qk_norm_forward", [sq] + [vp] * 8 + [vp], i32),
            ("qk_norm_backward", [sq] + [vp] * 12 + [vp, sz, vp], i32),
            ("kv_write", [sc] + [vp] * 9 + [vp], i32),
            ("kv_read", [sc] + [vp] * 9 + [vp], i32),
            ("attn_decode_workspace_bytes", [sd], sz),
            ("attn_decode", [sd] + [vp] * 8 + [vp, sz, vp], i32)):
        f = getattr(L, name)
        f.argtypes, f.restype = args, res
    _LIB = L
    return L


def status_text(status):
    return lib().wkv7_status_string(status).decode()


def check(func, status):
    if status != WKV7_OK:
        raise Wkv7Error(func, status, status_text(status))
