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
    if stream is None and index == torch.cuda.current_device():
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
    if t is None or t.shape != shape or t.dtype != dtype or not t.is_cuda or t.get_device() != index \
            or not t.is_contiguous():
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
