"""Thin torch-facing binding of the libwkv7 C ABI.

Argument marshalling only: torch allocates device memory and supplies the
stream; every step of the recurrence runs in the library's HIP kernels.
Names mirror the C entry points (include/wkv7.h).
"""
import ctypes
import functools

import torch

from . import _lib

_VEC_DTYPES = {torch.float32: _lib.WKV7_F32, torch.bfloat16: _lib.WKV7_BF16}


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _on(stream):
    """Allocate the buffers a call creates on the stream its kernels run on,
    so that the caching allocator does not hand their memory to other work
    before those kernels are done with it."""
    return torch.cuda.stream(stream) if stream is not None else _Nothing()


class _Nothing:
    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_ALGOS = {"auto": _lib.WKV7_ALGO_AUTO, "scan": _lib.WKV7_ALGO_SCAN,
          "chunked": _lib.WKV7_ALGO_CHUNKED}


def make_shape(B, T, H, N, dtype=torch.float32, chunk=64, algo="auto", fused=False):
    return _lib.Shape(B, T, H, N, _VEC_DTYPES[dtype], chunk, _ALGOS[algo],
                      _lib.WKV7_FUSED_INPUTS if fused else 0)


def _check_vecs(names, tensors):
    ref = tensors[0]
    if ref.dim() != 4:
        raise ValueError(f"{names[0]} must be [B, T, H, N]")
    if ref.dtype not in _VEC_DTYPES:
        raise ValueError(f"{names[0]}: dtype {ref.dtype} not supported")
    for n, t in zip(names, tensors):
        if t.shape != ref.shape or t.dtype != ref.dtype:
            raise ValueError(f"{n}: shape/dtype must match {names[0]}")
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous device tensor")
    return tuple(ref.shape), ref.dtype


def _check_state(name, t, B, H, N):
    if t is None:
        return
    if t.shape != (B, H, N, N) or t.dtype != torch.float32 or not t.is_cuda \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 device tensor [B, H, N, N]")


def wkv7_checkpoint_bytes(B, T, H, N, dtype=torch.float32, chunk=64):
    sh = make_shape(B, T, H, N, dtype, chunk)
    return _lib.lib().wkv7_checkpoint_bytes(ctypes.byref(sh))


def wkv7_backward_workspace_bytes(B, T, H, N, dtype=torch.float32, chunk=64, ckpt_provided=True):
    sh = make_shape(B, T, H, N, dtype, chunk)
    return _lib.lib().wkv7_backward_workspace_bytes(ctypes.byref(sh), int(bool(ckpt_provided)))


def wkv7_forward(r, w, k, v, a, b, s0=None, *, chunk=64, want_y=True, want_sT=True,
                 want_ckpt=False, stream=None, out=None, fused=False):
    """Run the forward scan.  Returns (y, sT, ckpt); unwanted outputs are None.

    fused=True (WKV7_FUSED_INPUTS): w, a, b carry omega, kk and the gate, and
    the library forms w = exp(-exp(-0.5) sigmoid(omega)), a = -kk, b = kk gate.

    ckpt is the flat fp32 checkpoint record (states every `chunk` steps, then
    the per-step sa) that wkv7_backward consumes.

    ``out`` may supply preallocated (y, sT, ckpt) tensors (None entries are
    allocated when wanted)."""
    (B, T, H, N), dt = _check_vecs("rwkvab", (r, w, k, v, a, b))
    _check_state("s0", s0, B, H, N)
    dev = r.device
    y, sT, ckpt = out if out is not None else (None, None, None)
    with _on(stream):
        if want_y and y is None:
            y = torch.empty((B, T, H, N), device=dev, dtype=torch.float32)
        if want_sT and sT is None:
            sT = torch.empty((B, H, N, N), device=dev, dtype=torch.float32)
        if want_ckpt and ckpt is None:
            ckpt = torch.empty(wkv7_checkpoint_bytes(B, T, H, N, dt, chunk) // 4, device=dev,
                               dtype=torch.float32)
    sh = make_shape(B, T, H, N, dt, chunk, fused=fused)
    rc = _lib.lib().wkv7_forward(ctypes.byref(sh), *map(_ptr, (r, w, k, v, a, b, s0)),
                                 _ptr(y if want_y else None), _ptr(sT if want_sT else None),
                                 _ptr(ckpt if want_ckpt else None), _stream(stream))
    _lib.check("wkv7_forward", rc)
    return (y if want_y else None), (sT if want_sT else None), (ckpt if want_ckpt else None)


def wkv7_backward(r, w, k, v, a, b, dy, s0=None, dsT=None, ckpt=None, *, chunk=64,
                  want_ds0=True, workspace=None, stream=None, out=None, algo="auto",
                  fused=False):
    """Run the reverse scan.  Returns dict(dr, dw, dk, dv, da, db, ds0).

    algo: "auto", "scan" or "chunked" (wkv7_algo).  fused=True: the inputs
    as for wkv7_forward(fused=True), and dw, da, db hold d omega, d kk and
    d gate."""
    (B, T, H, N), dt = _check_vecs("rwkvab dy", (r, w, k, v, a, b, dy))
    _check_state("s0", s0, B, H, N)
    _check_state("dsT", dsT, B, H, N)
    dev = r.device
    names = ("dr", "dw", "dk", "dv", "da", "db")
    grads = dict(out) if out is not None else {}
    need = wkv7_backward_workspace_bytes(B, T, H, N, dt, chunk, ckpt is not None)
    with _on(stream):
        for n in names:
            if grads.get(n) is None:
                grads[n] = torch.empty((B, T, H, N), device=dev, dtype=torch.float32)
        if want_ds0 and grads.get("ds0") is None:
            grads["ds0"] = torch.empty((B, H, N, N), device=dev, dtype=torch.float32)
        if workspace is None and need > 0:
            workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    if not want_ds0:
        grads["ds0"] = None
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    sh = make_shape(B, T, H, N, dt, chunk, algo, fused=fused)
    rc = _lib.lib().wkv7_backward(
        ctypes.byref(sh), *map(_ptr, (r, w, k, v, a, b, s0, dy, dsT, ckpt)),
        *map(_ptr, (grads[n] for n in names)), _ptr(grads["ds0"]),
        _ptr(workspace), ws_bytes, _stream(stream))
    _lib.check("wkv7_backward", rc)
    return grads


def wkv7_backward_noalloc(r, w, k, v, a, b, dy, s0=None, dsT=None, ckpt=None, *, out,
                          chunk=64, stream=None, algo="auto", fused=False):
    """wkv7_backward with the library's own fixed device workspace
    (WKV7_NOALLOC_SCRATCH_BYTES per GPU) instead of a caller workspace; the
    caller supplies every output in `out` (dict dr, dw, dk, dv, da, db and
    optionally ds0), so nothing is allocated.  Returns `out`."""
    (B, T, H, N), dt = _check_vecs("rwkvab dy", (r, w, k, v, a, b, dy))
    _check_state("s0", s0, B, H, N)
    _check_state("dsT", dsT, B, H, N)
    names = ("dr", "dw", "dk", "dv", "da", "db")
    for n in names:
        _check_f32(n, out[n], (B, T, H, N))
    if out.get("ds0") is not None:
        _check_f32("ds0", out["ds0"], (B, H, N, N))
    sh = make_shape(B, T, H, N, dt, chunk, algo, fused=fused)
    rc = _lib.lib().wkv7_backward_noalloc(
        ctypes.byref(sh), *map(_ptr, (r, w, k, v, a, b, s0, dy, dsT, ckpt)),
        *map(_ptr, (out[n] for n in names)), _ptr(out.get("ds0")), _stream(stream))
    _lib.check("wkv7_backward_noalloc", rc)
    return out


def _check_f32(name, t, shape):
    if t.shape != shape or t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous fp32 device tensor {list(shape)}")


def wkv7_epilogue_forward(y, r, k, v, g, ln_w, ln_b, r_k, *, stream=None, out=None):
    """Group norm, bonus and gate after the scan (wkv7_epilogue_forward):
    z = ((y - mean) rstd ln_w + ln_b + (sum r k r_k) v) g per (b, t, h)."""
    (B, T, H, N), dt = _check_vecs("rkvg", (r, k, v, g))
    _check_f32("y", y, (B, T, H, N))
    for n, p in (("ln_w", ln_w), ("ln_b", ln_b), ("r_k", r_k)):
        _check_f32(n, p, (H, N))
    with _on(stream):
        z = out if out is not None else torch.empty((B, T, H, N), device=y.device,
                                                    dtype=torch.float32)
    sh = make_shape(B, T, H, N, dt)
    rc = _lib.lib().wkv7_epilogue_forward(ctypes.byref(sh), *map(_ptr, (y, r, k, v, g, ln_w, ln_b, r_k, z)),
                                          _stream(stream))
    _lib.check("wkv7_epilogue_forward", rc)
    return z


def wkv7_epilogue_backward(dz, y, r, k, v, g, ln_w, ln_b, r_k, *, workspace=None, stream=None):
    """The epilogue's backward: dict(dy, dg, dr, dk, dv, dln_w, dln_b, dr_k);
    dr, dk, dv are the bonus term's shares (added to the scan's by the caller)."""
    (B, T, H, N), dt = _check_vecs("rkvg", (r, k, v, g))
    _check_f32("y", y, (B, T, H, N))
    _check_f32("dz", dz, (B, T, H, N))
    for n, p in (("ln_w", ln_w), ("ln_b", ln_b), ("r_k", r_k)):
        _check_f32(n, p, (H, N))
    dev = y.device
    sh = make_shape(B, T, H, N, dt)
    need = _lib.lib().wkv7_epilogue_workspace_bytes(ctypes.byref(sh))
    with _on(stream):
        out = {n: torch.empty((B, T, H, N), device=dev, dtype=torch.float32)
               for n in ("dy", "dg", "dr", "dk", "dv")}
        for n in ("dln_w", "dln_b", "dr_k"):
            out[n] = torch.empty((H, N), device=dev, dtype=torch.float32)
        if workspace is None and need > 0:
            workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = _lib.lib().wkv7_epilogue_backward(
        ctypes.byref(sh), *map(_ptr, (dz, y, r, k, v, g, ln_w, ln_b, r_k)),
        *map(_ptr, (out[n] for n in ("dy", "dg", "dr", "dk", "dv", "dln_w", "dln_b", "dr_k"))),
        _ptr(workspace), ws_bytes, _stream(stream))
    _lib.check("wkv7_epilogue_backward", rc)
    return out


# ---------------------------------------------------------------- RWKV-8 rho

def _rwkv8_dims(q, v, decay):
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q must be [B, H, T, L] and v [B, Hv, T, E]")
    B, H, T, L = q.shape
    Bv, Hv, Tv, E = v.shape
    if Bv != B or Tv != T or Hv not in (1, H) or tuple(decay.shape) != (H, L):
        raise ValueError(f"shapes q {tuple(q.shape)} v {tuple(v.shape)} decay {tuple(decay.shape)}")
    for n, t in (("q", q), ("v", v), ("decay", decay)):
        if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous fp32 device tensor")
    return B, H, T, L, Hv, E


def rwkv8_shape(B, T, H, Hv, L=64, E=64):
    return _lib.Rwkv8Shape(B, T, H, Hv, L, E)


def rwkv8_checkpoint_bytes(B, T, H, Hv, L=64, E=64):
    return _lib.lib().rwkv8_checkpoint_bytes(ctypes.byref(rwkv8_shape(B, T, H, Hv, L, E)))


def rwkv8_backward_workspace_bytes(B, T, H, Hv, L=64, E=64, ckpt_provided=True):
    return _lib.lib().rwkv8_backward_workspace_bytes(ctypes.byref(rwkv8_shape(B, T, H, Hv, L, E)),
                                                      int(bool(ckpt_provided)))


def rwkv8_forward(q, v, decay, rho0=None, norm0=None, *, want_y=True, want_state=True,
                  want_ckpt=False, stream=None, out=None):
    """The RWKV-8 rho / rho_norm forward (rwkv8_forward).  q [B, H, T, 64],
    v [B, Hv, T, 64], decay [H, 64], rho0 [B, H, 64, 64], norm0 [B, H, 64].
    Returns (y, rhoT, normT, ckpt); unwanted outputs are None."""
    B, H, T, L, Hv, E = _rwkv8_dims(q, v, decay)
    dev = q.device
    y, rT, nT, ck = out if out is not None else (None, None, None, None)
    with _on(stream):
        if want_y and y is None:
            y = torch.empty((B, H, T, E), device=dev, dtype=torch.float32)
        if want_state and rT is None:
            rT = torch.empty((B, H, L, E), device=dev, dtype=torch.float32)
            nT = torch.empty((B, H, L), device=dev, dtype=torch.float32)
        if want_ckpt and ck is None:
            ck = torch.empty(rwkv8_checkpoint_bytes(B, T, H, Hv, L, E) // 4, device=dev,
                             dtype=torch.float32)
    sh = rwkv8_shape(B, T, H, Hv, L, E)
    rc = _lib.lib().rwkv8_forward(ctypes.byref(sh), *map(_ptr, (q, v, decay, rho0, norm0)),
                                  _ptr(y if want_y else None), _ptr(rT if want_state else None),
                                  _ptr(nT if want_state else None), _ptr(ck if want_ckpt else None),
                                  _stream(stream))
    _lib.check("rwkv8_forward", rc)
    return ((y if want_y else None), (rT if want_state else None), (nT if want_state else None),
            (ck if want_ckpt else None))


def rwkv8_backward(q, v, decay, dy, rho0=None, norm0=None, drhoT=None, dnormT=None, ckpt=None, *,
                   want_state_grads=True, workspace=None, stream=None, out=None):
    """The RWKV-8 rho / rho_norm backward (rwkv8_backward).  Returns dict dq,
    dv, ddecay, drho0, dnorm0 (the last two None when not wanted)."""
    B, H, T, L, Hv, E = _rwkv8_dims(q, v, decay)
    dev = q.device
    g = dict(out) if out is not None else {}
    need = rwkv8_backward_workspace_bytes(B, T, H, Hv, L, E, ckpt is not None)
    with _on(stream):
        shapes = {"dq": (B, H, T, L), "dv": (B, Hv, T, E), "ddecay": (H, L)}
        if want_state_grads:
            shapes.update(drho0=(B, H, L, E), dnorm0=(B, H, L))
        for n, shp in shapes.items():
            if g.get(n) is None:
                g[n] = torch.empty(shp, device=dev, dtype=torch.float32)
        if workspace is None and need > 0:
            workspace = torch.empty(need, device=dev, dtype=torch.uint8)
    if not want_state_grads:
        g["drho0"] = g["dnorm0"] = None
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    sh = rwkv8_shape(B, T, H, Hv, L, E)
    rc = _lib.lib().rwkv8_backward(
        ctypes.byref(sh), *map(_ptr, (q, v, decay, rho0, norm0, dy, drhoT, dnormT, ckpt)),
        *map(_ptr, (g["dq"], g["dv"], g["ddecay"], g["drho0"], g["dnorm0"])),
        _ptr(workspace), ws_bytes, _stream(stream))
    _lib.check("rwkv8_backward", rc)
    return g


# ------------------------------------------------------ the gated delta rule

# The calls below are also made for single tokens, where their own host time is
# what a step waits for: plain integers for pointers, one look-up per shape and
# no context managers unless the caller's device or stream is not the current one.

def _raw_stream(index):
    """The handle of a device's current stream."""
    return torch._C._cuda_getCurrentRawStream(index)


def _launch(name, index, stream, call):
    """call(stream handle) with the device of the tensors as the current one and
    ``stream``, if given, as its stream (also for what it allocates)."""
    if stream is None and index == torch._C._cuda_getDevice():
        return call(_raw_stream(index))
    if stream is not None and stream.device.index != index:
        raise ValueError(f"{name}: the stream is on {stream.device}, the tensors on cuda:{index}")
    with torch.cuda.device(index), _on(stream):
        return call(_raw_stream(index))


def _at(t):
    return None if t is None else t.data_ptr()


def _check_like(name, t, shape, dtype, index, optional=False):
    if t is None and optional:
        return
    # (the device of a tensor that is not on one is -1)
    if t is None or t.shape != shape or t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on cuda:{index}")


def _workspace(name, workspace, need, index):
    """The workspace to pass on (the caller's, or one of `need` bytes), its
    address and its size."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, device=index, dtype=torch.uint8)
        return workspace, workspace.data_ptr(), need
    if not workspace.is_cuda or workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"{name}: workspace must be a contiguous tensor on cuda:{index}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _aligned(*tensors):
    """The tensors, those off the library's 16-byte alignment copied (on the
    current stream): slices of slots, starts, g or beta begin anywhere."""
    return [t if t is None or t.data_ptr() % 16 == 0 else t.clone() for t in tensors]


def _output(name, t, shape, dtype, index):
    """A caller's output, checked, or a new one."""
    if t is None:
        return torch.empty(shape, device=index, dtype=dtype)
    _check_like(name, t, shape, dtype, index)
    return t


def gdr_shape(B, T, Hk, Hv, K, V, dtype=torch.float32, nseq=0, norm_qk=False, scale=None):
    if scale is None:
        scale = K ** -0.5 if K > 0 else 1.0   # the library refuses other K
    return _lib.GdrShape(B, T, Hk, Hv, K, V, nseq, _VEC_DTYPES[dtype],
                         _lib.GDR_NORM_QK if norm_qk else 0, scale)


@functools.lru_cache(maxsize=256)
def _gdr_sizes(*key):
    """A shape for the library, and the bytes of its record and workspaces."""
    L, sh = _lib.lib(), gdr_shape(*key)
    r = ctypes.byref(sh)
    return sh, r, L.gdr_checkpoint_bytes(r), L.gdr_forward_workspace_bytes(r), \
        (L.gdr_backward_workspace_bytes(r, 0), L.gdr_backward_workspace_bytes(r, 1))


def gdr_checkpoint_bytes(B, T, Hk, Hv, K, V, dtype=torch.float32, nseq=0):
    return _lib.lib().gdr_checkpoint_bytes(ctypes.byref(gdr_shape(B, T, Hk, Hv, K, V, dtype, nseq)))


def gdr_forward_workspace_bytes(B, T, Hk, Hv, K, V, dtype=torch.float32, nseq=0):
    return _lib.lib().gdr_forward_workspace_bytes(
        ctypes.byref(gdr_shape(B, T, Hk, Hv, K, V, dtype, nseq)))


def gdr_backward_workspace_bytes(B, T, Hk, Hv, K, V, dtype=torch.float32, nseq=0, ckpt_provided=True):
    return _lib.lib().gdr_backward_workspace_bytes(
        ctypes.byref(gdr_shape(B, T, Hk, Hv, K, V, dtype, nseq)), int(bool(ckpt_provided)))


def _gdr_dims(q, k, v, g, beta, seq_starts, scale, norm_qk):
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q must be [B, T, Hk, K] and v [B, T, Hv, V]")
    dt = q.dtype
    if dt not in _VEC_DTYPES:
        raise ValueError(f"q: dtype {dt} not supported")
    if not q.is_cuda:
        raise ValueError("q must be a device tensor")
    qs, ys, at = q.shape, v.shape, q.get_device()
    B, T, Hk, K = qs
    Hv, V = ys[2], ys[3]
    if Hk == 0 or Hv % Hk != 0:
        raise ValueError(f"v has {Hv} heads: not a multiple of q's {Hk}")
    gs = (B, T, Hv)
    _check_like("q", q, qs, dt, at)
    _check_like("k", k, qs, dt, at)
    _check_like("v", v, (B, T, Hv, V), dt, at)
    _check_like("g", g, gs, torch.float32, at)
    _check_like("beta", beta, gs, torch.float32, at)
    nseq = 0
    if seq_starts is not None:
        nseq = seq_starts.numel() - 1
        if B != 1 or nseq < 1:
            raise ValueError("seq_starts needs B = 1 and at least two entries")
        _check_like("seq_starts", seq_starts, (nseq + 1,), torch.int32, at)
    return (B, T, Hk, Hv, K, V, dt, nseq, bool(norm_qk), None if scale is None else float(scale)), ys, (nseq or B, Hv, V, K), at


def gdr_forward(q, k, v, g, beta, s0=None, *, seq_starts=None, scale=None, norm_qk=False, want_y=True,
                want_sT=True, want_ckpt=False, workspace=None, stream=None, out=None):
    """The gated delta rule over whole sequences (gdr_forward):
    S_t = exp(g_t) S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,
    y_t = scale S_t q_t.  Returns (y, sT, ckpt); unwanted outputs are None.

    q, k [B, T, Hk, K], v [B, T, Hv, V] fp32 or bf16; g (log decay, <= 0) and
    beta [B, T, Hv] fp32; s0 [sequences, Hv, V, K] fp32 or None.  scale
    defaults to K ** -0.5.  norm_qk normalises q and k over K first.

    seq_starts (int32, on the device) packs sequences end to end into B = 1:
    sequence s is tokens seq_starts[s] .. seq_starts[s + 1] - 1.  Rows of y
    outside every sequence are not written.  No output may overlap an input.
    (A single long document is faster as a row, without seq_starts.)

    ckpt is the record gdr_backward consumes.  ``out`` may supply (y, sT,
    ckpt) tensors (None entries are allocated when wanted)."""
    key, ys, ss, at = _gdr_dims(q, k, v, g, beta, seq_starts, scale, norm_qk)
    _, sh, ck_bytes, need, _ = _gdr_sizes(*key)
    f32 = torch.float32
    _check_like("s0", s0, ss, f32, at, optional=True)
    y, sT, ckpt = out if out is not None else (None, None, None)

    def call(st):
        y_ = _output("y", y, ys, q.dtype, at) if want_y else None
        sT_ = _output("sT", sT, ss, f32, at) if want_sT else None
        ckpt_ = _output("ckpt", ckpt, (ck_bytes // 4,), f32, at) if want_ckpt else None
        ws, wp, wb = _workspace("gdr_forward", workspace, need, at)
        g_, beta_, starts = _aligned(g, beta, seq_starts)
        rc = _lib.lib().gdr_forward(sh, *map(_at, (q, k, v, g_, beta_, s0, starts, y_, sT_, ckpt_)), wp, wb, st)
        _lib.check("gdr_forward", rc)
        return y_, sT_, ckpt_

    return _launch("gdr_forward", at, stream, call)


def gdr_backward(q, k, v, g, beta, dy, s0=None, dsT=None, ckpt=None, *, seq_starts=None, scale=None,
                 norm_qk=False, want_ds0=True, workspace=None, stream=None, out=None):
    """The gradients of gdr_forward (gdr_backward), with the same inputs and
    options.  Returns dict(dq, dk, dv, dg, dbeta, ds0): dq, dk, dv in the
    inputs' type, the others fp32; ds0 None when not wanted."""
    key, ys, ss, at = _gdr_dims(q, k, v, g, beta, seq_starts, scale, norm_qk)
    _, sh, ck_bytes, _, need = _gdr_sizes(*key)
    f32 = torch.float32
    _check_like("dy", dy, ys, q.dtype, at)
    _check_like("s0", s0, ss, f32, at, optional=True)
    _check_like("dsT", dsT, ss, f32, at, optional=True)
    _check_like("ckpt", ckpt, (ck_bytes // 4,), f32, at, optional=True)
    grads = dict(out) if out is not None else {}

    def call(st):
        for n, like in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta)):
            grads[n] = _output(n, grads.get(n), like.shape, like.dtype, at)
        grads["ds0"] = _output("ds0", grads.get("ds0"), ss, f32, at) if want_ds0 else None
        ws, wp, wb = _workspace("gdr_backward", workspace, need[ckpt is not None], at)
        g_, beta_, starts = _aligned(g, beta, seq_starts)
        rc = _lib.lib().gdr_backward(
            sh, *map(_at, (q, k, v, g_, beta_, s0, starts, dy, dsT, ckpt)),
            *(_at(grads[n]) for n in ("dq", "dk", "dv", "dg", "dbeta", "ds0")), wp, wb, st)
        _lib.check("gdr_backward", rc)
        return grads

    return _launch("gdr_backward", at, stream, call)


def gdr_decode(q, k, v, g, beta, state, slots=None, *, scale=None, norm_qk=False, stream=None, out=None):
    """The recurrent form for a few tokens (gdr_decode): runs the T tokens of
    each row from and back into ``state`` [pool, Hv, V, K] fp32, in place, and
    returns y [B, T, Hv, V].  slots (int32 [B], on the device) names each
    row's state, None is row b = state b.  A row with a slot outside the pool,
    or with an earlier row's slot, is skipped: its y is left as it was."""
    key, ys, ss, at = _gdr_dims(q, k, v, g, beta, None, scale, norm_qk)
    if state.dim() != 4:
        raise ValueError("state must be [pool, Hv, V, K]")
    pool = state.shape[0]
    _check_like("state", state, (pool,) + ss[1:], torch.float32, at)
    if slots is not None:
        _check_like("slots", slots, (ys[0],), torch.int32, at)
    elif pool < ys[0]:
        raise ValueError(f"state holds {pool} states for {ys[0]} rows")
    sh = _gdr_sizes(*key)[1]

    def call(st):
        y = _output("y", out, ys, q.dtype, at)
        g_, beta_, slots_ = _aligned(g, beta, slots)
        rc = _lib.lib().gdr_decode(sh, q.data_ptr(), k.data_ptr(), v.data_ptr(), g_.data_ptr(), beta_.data_ptr(),
                                   state.data_ptr(), pool, _at(slots_), y.data_ptr(), st)
        _lib.check("gdr_decode", rc)
        return y

    return _launch("gdr_decode", at, stream, call)


@functools.lru_cache(maxsize=256)
def _epilogue_sizes(*key):
    sh = _lib.GdrEpilogueShape(*key)
    r = ctypes.byref(sh)
    return sh, r, _lib.lib().gdr_epilogue_workspace_bytes(r)


def gdr_epilogue_workspace_bytes(rows, H, N, Hw=1, dtype=torch.float32):
    """Of gdr_epilogue_backward: ``rows`` tokens of H heads of N, weights for
    Hw heads (1 or H)."""
    return _epilogue_sizes(rows, H, N, Hw, _VEC_DTYPES[dtype], 0, 1e-6)[2]


def _gdr_epilogue_dims(y, gate, w, eps):
    if y.dim() != 4 or w.dim() != 2:
        raise ValueError("y must be [B, T, H, N] and w [1 or H, N]")
    dt = y.dtype
    if dt not in _VEC_DTYPES:
        raise ValueError(f"y: dtype {dt} not supported")
    if not y.is_cuda:
        raise ValueError("y must be a device tensor")
    ys, at = y.shape, y.get_device()
    B, T, H, N = ys
    Hw = w.shape[0]
    if Hw not in (1, H):
        raise ValueError(f"w has {Hw} heads: 1 or {H}")
    _check_like("y", y, ys, dt, at)
    _check_like("gate", gate, ys, dt, at)
    _check_like("w", w, (Hw, N), torch.float32, at)
    return _epilogue_sizes(B * T, H, N, Hw, _VEC_DTYPES[dt], 0, float(eps)), ys, at


def gdr_epilogue_forward(y, gate, w, *, eps=1e-6, stream=None, out=None):
    """The gated norm after the scan (gdr_epilogue_forward), per head:
    z = y / sqrt(mean(y^2) + eps) * w * gate * sigmoid(gate).
    y, gate [B, T, H, N] fp32 or bf16, w [1 or H, N] fp32."""
    (_, sh, _), ys, at = _gdr_epilogue_dims(y, gate, w, eps)

    def call(st):
        z = _output("z", out, ys, y.dtype, at)
        rc = _lib.lib().gdr_epilogue_forward(sh, y.data_ptr(), gate.data_ptr(), w.data_ptr(), z.data_ptr(), st)
        _lib.check("gdr_epilogue_forward", rc)
        return z

    return _launch("gdr_epilogue_forward", at, stream, call)


def gdr_epilogue_backward(dz, y, gate, w, *, eps=1e-6, workspace=None, stream=None, out=None):
    """The epilogue's gradients: dict(dy, dgate, dw), dw fp32 like w."""
    (_, sh, need), ys, at = _gdr_epilogue_dims(y, gate, w, eps)
    _check_like("dz", dz, ys, y.dtype, at)
    grads = dict(out) if out is not None else {}

    def call(st):
        for n, like in (("dy", y), ("dgate", gate), ("dw", w)):
            grads[n] = _output(n, grads.get(n), like.shape, like.dtype, at)
        ws, wp, wb = _workspace("gdr_epilogue_backward", workspace, need, at)
        rc = _lib.lib().gdr_epilogue_backward(sh, *map(_at, (dz, y, gate, w)),
                                              *(_at(grads[n]) for n in ("dy", "dgate", "dw")), wp, wb, st)
        _lib.check("gdr_epilogue_backward", rc)
        return grads

    return _launch("gdr_epilogue_backward", at, stream, call)


# --------------------------------------------------------- the residual norm

@functools.lru_cache(maxsize=256)
def _norm_sizes(*key):
    sh = _lib.ResidualNormShape(*key)
    r = ctypes.byref(sh)
    return sh, r, _lib.lib().residual_norm_workspace_bytes(r)


def residual_norm_workspace_bytes(rows, D, dtype=torch.float32):
    """Of residual_norm_backward: ``rows`` rows of D."""
    return _norm_sizes(rows, D, _VEC_DTYPES[dtype], 0, 1e-6)[2]


def _norm_dims(x, eps):
    if x.dim() < 1 or x.dtype not in _VEC_DTYPES or not x.is_cuda or not x.is_contiguous():
        raise ValueError("the residual stream must be a contiguous fp32 or bf16 device tensor [..., D]")
    D = x.shape[-1]
    if D == 0:
        raise ValueError("the residual stream has rows of no entries")
    return _norm_sizes(x.numel() // D, D, _VEC_DTYPES[x.dtype], 0, float(eps)), D, x.get_device()


def residual_norm_forward(x, y, w, scale=None, *, eps=1e-6, want_x_out=True, stream=None, out=None):
    """The residual sum and the norm before the next block
    (residual_norm_forward): x_out = x + scale * y, h = x_out /
    sqrt(mean(x_out^2) + eps) * w over the last axis.  Returns (x_out, h).
    x, y [..., D] fp32 or bf16 (y None: x_out = x); w, scale [D] fp32.
    ``out`` may supply (x_out, h); x_out may be x itself."""
    (_, sh, _), D, at = _norm_dims(x, eps)
    f32, xs, dt = torch.float32, x.shape, x.dtype
    _check_like("y", y, xs, dt, at, optional=True)
    _check_like("w", w, (D,), f32, at)
    _check_like("scale", scale, (D,), f32, at, optional=True)
    if scale is not None and y is None:
        raise ValueError("scale needs y")
    xo, h = out if out is not None else (None, None)

    def call(st):
        xo_ = _output("x_out", xo, xs, dt, at) if want_x_out else None
        h_ = _output("h", h, xs, dt, at)
        rc = _lib.lib().residual_norm_forward(sh, x.data_ptr(), _at(y), _at(scale), w.data_ptr(), _at(xo_),
                                              h_.data_ptr(), st)
        _lib.check("residual_norm_forward", rc)
        return xo_, h_

    return _launch("residual_norm_forward", at, stream, call)


def residual_norm_backward(dh, dx_out, x_out, w, y=None, scale=None, *, eps=1e-6, workspace=None,
                           stream=None, out=None):
    """The gradients of residual_norm_forward from those of h and x_out
    (dx_out None: zeros), with x_out as it was stored: dict(dx, dy, dw,
    dscale).  Without a scale, dx is the gradient of y too, and dy and dscale
    are None; with one, y is needed as well.  dx may be dx_out itself."""
    (_, sh, need), D, at = _norm_dims(x_out, eps)
    dt, f32, xs = x_out.dtype, torch.float32, x_out.shape
    _check_like("dh", dh, xs, dt, at)
    _check_like("dx_out", dx_out, xs, dt, at, optional=True)
    _check_like("w", w, (D,), f32, at)
    if (scale is None) != (y is None):
        raise ValueError("y and scale come together")
    scaled = scale is not None
    _check_like("scale", scale, (D,), f32, at, optional=True)
    _check_like("y", y, xs, dt, at, optional=True)
    grads = dict(out) if out is not None else {}

    def call(st):
        grads["dx"] = _output("dx", grads.get("dx"), xs, dt, at)
        grads["dw"] = _output("dw", grads.get("dw"), (D,), f32, at)
        grads["dy"] = _output("dy", grads.get("dy"), xs, dt, at) if scaled else None
        grads["dscale"] = _output("dscale", grads.get("dscale"), (D,), f32, at) if scaled else None
        ws, wp, wb = _workspace("residual_norm_backward", workspace, need, at)
        rc = _lib.lib().residual_norm_backward(
            sh, *map(_at, (dh, dx_out, x_out, y, scale, w)),
            *(_at(grads[n]) for n in ("dx", "dy", "dw", "dscale")), wp, wb, st)
        _lib.check("residual_norm_backward", rc)
        return grads

    return _launch("residual_norm_backward", at, stream, call)


# --------------------------------------------------------- softmax attention

def _token_stride(name, t, heads, D, dtype, index, B=None, T=None):
    """Checks [B, T, heads, D] with heads end to end and rows one after the
    other; returns the elements from a token to the next (0: contiguous)."""
    if t is None or t.dtype is not dtype or t.get_device() != index or t.dim() != 4:
        raise ValueError(f"{name} must be a {dtype} tensor [B, T, heads, D] on cuda:{index}")
    b, n, h, d = t.shape
    if d != D or h != heads or (B is not None and (b != B or n != T)):
        raise ValueError(f"{name} must be [{b if B is None else B}, {n if T is None else T}, {heads}, {D}]")
    if t.is_contiguous():
        return 0
    s = t.stride()
    step = s[1] if n > 1 else s[0] if b > 1 else 0
    if s[3] != 1 or (h > 1 and s[2] != D) or (b > 1 and s[0] != n * step) or step % 8 != 0 \
            or (b * n > 1 and step < h * D):
        raise ValueError(f"{name}: a token's heads must lie end to end, tokens and rows at one stride, a multiple of 8")
    return step


def _heads(name, q, k):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B, T, Hq, D] and k [B, T, Hk, D]")
    if q.dtype not in _VEC_DTYPES:
        raise ValueError(f"{name}: dtype {q.dtype} not supported")
    if not q.is_cuda:
        raise ValueError("q must be a device tensor")


def _int32(name, t, shape, index):
    if t is None or t.dtype is not torch.int32 or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor {list(shape)} on cuda:{index}")


def _output_like(name, t, like, index):
    """A caller's output, checked, or a new one, of another tensor's shape and
    type (which takes half the time of one from a shape)."""
    if t is None:
        return torch.empty_like(like, memory_format=torch.contiguous_format)
    _check_like(name, t, like.shape, like.dtype, index)
    return t


@functools.lru_cache(maxsize=256)
def _attn_sizes(*key):
    sh = _lib.AttnShape(*key)
    r = ctypes.byref(sh)
    return sh, r, _lib.lib().attn_record_bytes(r), _lib.lib().attn_backward_workspace_bytes(r)


def _attn_key(B, T, Hq, Hk, D, dtype, nseq=0, strides=(0, 0, 0), scale=None):
    if scale is None:
        scale = D ** -0.5 if D > 0 else 1.0   # the library refuses other D
    return (B, T, Hq, Hk, D, nseq, *strides, _VEC_DTYPES[dtype], 0, float(scale))


def attn_record_bytes(B, T, Hq, Hk, D, dtype=torch.bfloat16, nseq=0):
    return _attn_sizes(*_attn_key(B, T, Hq, Hk, D, dtype, nseq))[2]


def attn_backward_workspace_bytes(B, T, Hq, Hk, D, dtype=torch.bfloat16, nseq=0):
    return _attn_sizes(*_attn_key(B, T, Hq, Hk, D, dtype, nseq))[3]


def _attn_dims(q, k, v, seq_starts, scale):
    _heads("q", q, k)
    dt, at = q.dtype, q.get_device()
    B, T, Hq, D = q.shape
    Hk = k.shape[2]
    if Hk == 0 or Hq == 0 or Hq % Hk != 0:
        raise ValueError(f"q has {Hq} heads: not a multiple of k's {Hk}")
    strides = (_token_stride("q", q, Hq, D, dt, at), _token_stride("k", k, Hk, D, dt, at, B, T),
               _token_stride("v", v, Hk, D, dt, at, B, T))
    nseq = 0
    if seq_starts is not None:
        nseq = seq_starts.numel() - 1
        if B != 1 or nseq < 1:
            raise ValueError("seq_starts needs B = 1 and at least two entries")
        _int32("seq_starts", seq_starts, (nseq + 1,), at)
    return _attn_sizes(*_attn_key(B, T, Hq, Hk, D, dt, nseq, strides, scale)), q.shape, at


def attn_forward(q, k, v, *, seq_starts=None, scale=None, want_lse=False, want_record=False, stream=None, out=None):
    """Causal softmax attention over whole sequences (attn_forward):
    y_i = sum over j <= i of exp(scale q_i . k_j - lse_i) v_j.  Returns
    (y, lse, record); unwanted outputs are None.

    q [B, T, Hq, D], k, v [B, T, Hk, D] fp32 or bf16, D 64 or 128, Hq a multiple
    of Hk; each may be part of a wider tensor (heads end to end, one stride from
    token to token).  scale defaults to D ** -0.5 and is positive.  lse
    [B, T, Hq] fp32.

    seq_starts (int32, on the device) packs sequences end to end into B = 1:
    sequence s is tokens seq_starts[s] .. seq_starts[s + 1] - 1.  Rows of y and
    lse outside every sequence are not written.  No output may overlap an input.

    attn_backward takes y, lse and (bf16; with fp32 there is none) record.
    ``out`` may supply (y, lse, record) tensors (None entries are allocated when
    wanted)."""
    (_, sh, _, _), ys, at = _attn_dims(q, k, v, seq_starts, scale)
    y, lse, rec = out if out is not None else (None, None, None)

    def call(st):
        y_ = _output_like("y", y, q, at)
        lse_ = _output("lse", lse, ys[:3], torch.float32, at) if want_lse else None
        rec_ = _output_like("record", rec, q, at) if want_record and q.dtype == torch.bfloat16 else None
        rc = _lib.lib().attn_forward(sh, *map(_at, (q, k, v, seq_starts, y_, lse_, rec_)), st)
        _lib.check("attn_forward", rc)
        return y_, lse_, rec_

    return _launch("attn_forward", at, stream, call)


def attn_backward(q, k, v, y, lse, dy, record=None, *, seq_starts=None, scale=None, workspace=None, stream=None,
                  out=None):
    """The gradients of attn_forward (attn_backward), with the same inputs and
    options and its y, lse and record, and dy, contiguous: dict(dq, dk, dv),
    contiguous, dk and dv summed over the query heads that read them.  Without the record y's own
    rounding to bf16 enters dq and dk."""
    (_, sh, _, need), ys, at = _attn_dims(q, k, v, seq_starts, scale)
    _check_like("y", y, ys, q.dtype, at)
    _check_like("dy", dy, ys, q.dtype, at)
    _check_like("lse", lse, ys[:3], torch.float32, at)
    if record is not None and q.dtype != torch.bfloat16:
        raise ValueError("record is for bf16 inputs")
    _check_like("record", record, ys, q.dtype, at, optional=True)
    grads = dict(out) if out is not None else {}

    def call(st):
        for n, like in (("dq", q), ("dk", k), ("dv", v)):
            grads[n] = _output_like(n, grads.get(n), like, at)
        ws, wp, wb = _workspace("attn_backward", workspace, need, at)
        rc = _lib.lib().attn_backward(sh, *map(_at, (q, k, v, seq_starts, y, lse, record, dy)),
                                      *(_at(grads[n]) for n in ("dq", "dk", "dv")), wp, wb, st)
        _lib.check("attn_backward", rc)
        return grads

    return _launch("attn_backward", at, stream, call)


# ----------------------------------------- the norm and rotation before it

@functools.lru_cache(maxsize=256)
def _qk_norm_sizes(*key):
    sh = _lib.QkNormShape(*key)
    r = ctypes.byref(sh)
    return sh, r, _lib.lib().qk_norm_workspace_bytes(r)


def qk_norm_workspace_bytes(B, T, Hq, Hk, D, dtype=torch.bfloat16):
    """Of qk_norm_backward with weights."""
    return _qk_norm_sizes(B, T, Hq, Hk, D, 0, 0, 0, _VEC_DTYPES[dtype], 0, 1e-6)[2]


def _qk_norm_dims(q, k, wq, wk, theta, positions, eps, interleaved):
    _heads("q", q, k)
    dt, at = q.dtype, q.get_device()
    B, T, Hq, D = q.shape
    Hk = k.shape[2]
    strides = (_token_stride("q", q, Hq, D, dt, at), _token_stride("k", k, Hk, D, dt, at, B, T))
    if (wq is None) != (wk is None):
        raise ValueError("wq and wk come together")
    _check_like("wq", wq, (D,), torch.float32, at, optional=True)
    _check_like("wk", wk, (D,), torch.float32, at, optional=True)
    R = 0
    if theta is not None:
        R = 2 * theta.numel()
        if theta.numel() == 0 or R > D:
            raise ValueError(f"theta must have 1 to {D // 2} entries")
        _check_like("theta", theta, (R // 2,), torch.float32, at)
    if positions is not None:
        _int32("positions", positions, (B, T), at)
    key = (B, T, Hq, Hk, D, R, *strides, _VEC_DTYPES[dt], _lib.QK_NORM_INTERLEAVED if interleaved else 0, float(eps))
    return _qk_norm_sizes(*key), at


def qk_norm_forward(q, k, wq=None, wk=None, theta=None, positions=None, *, eps=1e-6, interleaved=False, stream=None,
                    out=None):
    """The norm of queries and keys per head and their rotation, in one pass
    (qk_norm_forward): n = x / sqrt(mean(x^2) + eps) * w over a head's D
    entries (no weights: n = x), then the pairs of its first R entries turned by
    positions * theta (no theta: none).  Returns (q', k'), contiguous.

    q [B, T, Hq, D], k [B, T, Hk, D] fp32 or bf16, D 64 or 128, each may be part
    of a wider tensor; wq, wk [D], theta [R / 2] fp32, R a multiple of 16 up to
    D; positions int32 [B, T], by default 0 .. T - 1 in each row.  Pair i is
    (n[i], n[i + R / 2]), or with ``interleaved`` (n[2 i], n[2 i + 1]).  Angles
    are formed in fp64.  ``out`` may supply (q', k'); contiguous q and k
    themselves are allowed there."""
    (_, sh, _), at = _qk_norm_dims(q, k, wq, wk, theta, positions, eps, interleaved)
    qz, kz = out if out is not None else (None, None)

    def call(st):
        qz_ = _output_like("q'", qz, q, at)
        kz_ = _output_like("k'", kz, k, at)
        rc = _lib.lib().qk_norm_forward(sh, q.data_ptr(), k.data_ptr(), _at(wq), _at(wk), _at(theta), _at(positions),
                                        qz_.data_ptr(), kz_.data_ptr(), st)
        _lib.check("qk_norm_forward", rc)
        return qz_, kz_

    return _launch("qk_norm_forward", at, stream, call)


def qk_norm_backward(dqz, dkz, q, k, wq=None, wk=None, theta=None, positions=None, *, eps=1e-6, interleaved=False,
                     workspace=None, stream=None, out=None):
    """The gradients of qk_norm_forward from those of q' and k', with its
    inputs and options: dict(dq, dk, dwq, dwk), the weights' in fp32 and None
    without weights.  ``out`` may supply them; dq and dk may be dqz and dkz."""
    (_, sh, need), at = _qk_norm_dims(q, k, wq, wk, theta, positions, eps, interleaved)
    _check_like("dqz", dqz, q.shape, q.dtype, at)
    _check_like("dkz", dkz, k.shape, q.dtype, at)
    normed = wq is not None
    grads = dict(out) if out is not None else {}

    def call(st):
        grads["dq"] = _output_like("dq", grads.get("dq"), q, at)
        grads["dk"] = _output_like("dk", grads.get("dk"), k, at)
        for n, w in (("dwq", wq), ("dwk", wk)):
            grads[n] = _output_like(n, grads.get(n), w, at) if normed else None
        ws, wp, wb = _workspace("qk_norm_backward", workspace, need if normed else 0, at)
        rc = _lib.lib().qk_norm_backward(sh, *map(_at, (dqz, dkz, q, k, wq, wk, theta, positions)),
                                         *(_at(grads[n]) for n in ("dq", "dk", "dwq", "dwk")), wp, wb, st)
        _lib.check("qk_norm_backward", rc)
        return grads

    return _launch("qk_norm_backward", at, stream, call)


# ----------------------------------------------------------- the paged cache

_E4M3 = torch.float8_e4m3fn


def _cache_dims(k_pages, v_pages, table, lens, k_scale, v_scale, dtype, at):
    """Checks a cache against the type of the tokens; returns pages, Hk, page,
    D, rows, max_pages and the library's name of its type."""
    if k_pages.dim() != 4 or table.dim() != 2:
        raise ValueError("k_pages must be [pages, Hk, page, D] and table [rows, max_pages]")
    if k_pages.dtype not in (dtype, _E4M3):
        raise ValueError(f"k_pages: {k_pages.dtype} does not go with {dtype}: the same, or {_E4M3}")
    ps, kind = k_pages.shape, k_pages.dtype
    if k_pages.get_device() != at or not k_pages.is_contiguous():
        raise ValueError(f"k_pages must be a contiguous tensor on cuda:{at}")
    _check_like("v_pages", v_pages, ps, kind, at)
    rows, most = ts = table.shape
    _int32("table", table, ts, at)
    _int32("lens", lens, ts[:1], at)
    small = kind is _E4M3
    if small:
        _check_like("k_scale", k_scale, ps[:3], torch.float32, at)
        _check_like("v_scale", v_scale, ps[:3], torch.float32, at)
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale and v_scale are for an 8-bit cache")
    return (*ps, rows, most, _lib.KV_CACHE_E4M3 if small else _lib.KV_CACHE_SAME)


@functools.lru_cache(maxsize=256)
def _cache_shape(*key):
    sh = _lib.KvCacheShape(*key)
    return sh, ctypes.byref(sh)


def kv_write(k, v, k_pages, v_pages, table, lens, k_scale=None, v_scale=None, *, seq_starts=None, stream=None):
    """Writes new tokens' keys and values into their pages (kv_write), in place.

    k, v [B, T, Hk, D] fp32 or bf16 (each may be part of a wider tensor): the T
    last tokens of each of B rows, or with seq_starts (int32 [B + 1], on the
    device; k and v [1, tokens, Hk, D]) tokens seq_starts[r] .. seq_starts[r + 1]
    - 1 the last of row r.  Row r holds lens[r] tokens, the new ones among them
    (int32 [B]), in the pages table[r] (int32 [B, max_pages]), in order.
    k_pages, v_pages [pages, Hk, page, D] in k's type, or float8_e4m3fn with
    k_scale, v_scale [pages, Hk, page] fp32: each token's head is stored times
    448 / max|x|.  page is a power of two from 16 to 256.

    Tokens at positions below 0, past the table or in a page outside the pool
    are not written.  Two rows may share pages, but one place must not be written
    twice in a call."""
    if k.dim() != 4 or k.dtype not in _VEC_DTYPES or not k.is_cuda:
        raise ValueError("k must be an fp32 or bf16 device tensor [B, T, Hk, D]")
    at, dt = k.get_device(), k.dtype
    pages, Hk, page, D, rows, most, kind = _cache_dims(k_pages, v_pages, table, lens, k_scale, v_scale, dt, at)
    B, T = k.shape[:2]
    sk = _token_stride("k", k, Hk, D, dt, at)
    sv = _token_stride("v", v, Hk, D, dt, at, B, T)
    packed = _packed_rows(seq_starts, B, rows, at)
    _, sh = _cache_shape(rows, T, Hk, D, packed, pages, page, most, sk, sv, _VEC_DTYPES[dt], kind)

    def call(st):
        rc = _lib.lib().kv_write(sh, k.data_ptr(), v.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), _at(k_scale),
                                 _at(v_scale), table.data_ptr(), lens.data_ptr(), _at(seq_starts), st)
        _lib.check("kv_write", rc)

    return _launch("kv_write", at, stream, call)


def _packed_rows(seq_starts, B, rows, at):
    if seq_starts is None:
        if B != rows:
            raise ValueError(f"{B} rows of tokens for a table of {rows}")
        return 0
    if B != 1:
        raise ValueError("seq_starts needs B = 1")
    _int32("seq_starts", seq_starts, (rows + 1,), at)
    return 1


def kv_read(k_pages, v_pages, table, lens, k_scale=None, v_scale=None, *, T, seq_starts=None, dtype=None, stream=None,
            out=None):
    """The reverse of kv_write (kv_read): the T last tokens of each row, [rows,
    T, Hk, D], or with seq_starts the seq_starts[r + 1] - seq_starts[r] last ones
    of row r, end to end, [1, T, Hk, D] (rows outside every sequence are not
    written).  ``dtype`` is fp32 or bf16: the cache's own, or, by default bf16,
    what an 8-bit cache's values times their scales are rounded to.  Tokens
    that kv_write would not write are zeros.  Returns (k, v); ``out`` may supply
    them."""
    at = k_pages.get_device()
    if not k_pages.is_cuda:
        raise ValueError("k_pages must be a device tensor")
    if dtype is None:
        dtype = torch.bfloat16 if k_pages.dtype == _E4M3 else k_pages.dtype
    if dtype not in _VEC_DTYPES:
        raise ValueError(f"kv_read: dtype {dtype} not supported")
    if T < 0:
        raise ValueError("T is negative")
    pages, Hk, page, D, rows, most, kind = _cache_dims(k_pages, v_pages, table, lens, k_scale, v_scale, dtype, at)
    packed = _packed_rows(seq_starts, rows if seq_starts is None else 1, rows, at)
    shape = (1 if packed else rows, T, Hk, D)
    _, sh = _cache_shape(rows, T, Hk, D, packed, pages, page, most, 0, 0, _VEC_DTYPES[dtype], kind)
    k, v = out if out is not None else (None, None)

    def call(st):
        k_, v_ = _output("k", k, shape, dtype, at), _output("v", v, shape, dtype, at)
        rc = _lib.lib().kv_read(sh, *map(_at, (k_pages, v_pages, k_scale, v_scale, table, lens, seq_starts, k_, v_)), st)
        _lib.check("kv_read", rc)
        return k_, v_

    return _launch("kv_read", at, stream, call)


@functools.lru_cache(maxsize=256)
def _decode_sizes(*key):
    sh = _lib.AttnDecodeShape(*key)
    r = ctypes.byref(sh)
    return sh, r, _lib.lib().attn_decode_workspace_bytes(r)


def attn_decode_workspace_bytes(B, T, Hq, Hk, D, pages, page, max_pages, dtype=torch.bfloat16):
    return _decode_sizes(B, T, Hq, Hk, D, pages, page, max_pages, 0, _VEC_DTYPES[dtype], _lib.KV_CACHE_SAME, 1.0)[2]


def attn_decode(q, k_pages, v_pages, table, lens, k_scale=None, v_scale=None, *, scale=None, workspace=None,
                stream=None, out=None):
    """Attention of each row's T last tokens over the paged cache (attn_decode),
    which holds their keys and values already (kv_write); token t of row b sees
    the positions below lens[b] - (T - 1 - t).  Returns y [B, T, Hq, D].

    q [B, T, Hq, D] fp32 or bf16 (may be part of a wider tensor); the cache as
    for kv_write, in q's type or float8_e4m3fn.  scale defaults to D ** -0.5 and
    is positive.  Positions in a page outside the pool are seen by nobody; a
    token that sees nothing has y = 0."""
    if q.dim() != 4 or q.dtype not in _VEC_DTYPES or not q.is_cuda:
        raise ValueError("q must be an fp32 or bf16 device tensor [B, T, Hq, D]")
    at, dt = q.get_device(), q.dtype
    pages, Hk, page, D, rows, most, kind = _cache_dims(k_pages, v_pages, table, lens, k_scale, v_scale, dt, at)
    B, T, Hq, _ = q.shape
    if B != rows:
        raise ValueError(f"{B} rows of q for a table of {rows}")
    if Hk == 0 or Hq == 0 or Hq % Hk != 0:
        raise ValueError(f"q has {Hq} heads: not a multiple of the cache's {Hk}")
    sq = _token_stride("q", q, Hq, D, dt, at)
    if scale is None:
        scale = D ** -0.5 if D > 0 else 1.0
    _, sh, need = _decode_sizes(B, T, Hq, Hk, D, pages, page, most, sq, _VEC_DTYPES[dt], kind, float(scale))

    def call(st):
        y = _output_like("y", out, q, at)
        ws, wp, wb = _workspace("attn_decode", workspace, need, at)
        rc = _lib.lib().attn_decode(sh, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), _at(k_scale), _at(v_scale),
                                    table.data_ptr(), lens.data_ptr(), y.data_ptr(), wp, wb, st)
        _lib.check("attn_decode", rc)
        return y

    return _launch("attn_decode", at, stream, call)
