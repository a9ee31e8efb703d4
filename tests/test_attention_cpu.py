"""Softmax attention, the norm and rotation before it and the paged cache
without a GPU: the oracle against autograd, differences and closed forms; the
C ABI's exports, sizes and refusals (no call here launches a kernel)."""
import ctypes
import os
import re

import pytest
import torch

import linear_attention_rnn_wkv7_amd as pkg
import oracle.attention as R
from linear_attention_rnn_wkv7_amd import _lib, api

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, WORKSPACE = (_lib.WKV7_OK, _lib.WKV7_ERR_INVALID, _lib.WKV7_ERR_UNSUPPORTED,
                                       _lib.WKV7_ERR_WORKSPACE)


def rn(gen, *s):
    return torch.randn(s, generator=gen, dtype=torch.float64)


# ------------------------------------------------------------------ the oracle

@pytest.mark.parametrize("starts", [None, [0, 0, 1, 5, 7], [1, 4, 6]])
def test_oracle_attention_gradients(starts):
    B, T = (2, 5) if starts is None else (1, 7)
    gen = torch.Generator().manual_seed(1)
    q, k, v, dy = rn(gen, B, T, 4, 3), rn(gen, B, T, 2, 3), rn(gen, B, T, 2, 3), rn(gen, B, T, 4, 3)
    inside = torch.zeros(B, T, dtype=torch.bool)
    # the definition, as one masked softmax over the whole row
    place = torch.zeros(T, dtype=torch.long) - 1
    for i, (_, lo, hi) in enumerate(R._sequences(B, T, starts)):
        inside[:, lo:hi] = True
        place[lo:hi] = 0 if starts is None else i
    seen = (place[:, None] == place[None]) & torch.ones(T, T, dtype=torch.bool).tril() & (place[:, None] >= 0)
    a = [x.clone().requires_grad_() for x in (q, k, v)]
    s = 0.7 * torch.einsum("bihd,bjhd->bhij", a[0], a[1].repeat_interleave(2, 2))
    p = torch.softmax(s.masked_fill(~seen, -1e300), -1) * seen
    y = torch.einsum("bhij,bjhd->bihd", p, a[2].repeat_interleave(2, 2))
    want = torch.autograd.grad((y * dy).sum(), a)
    got = R.attention(q, k, v, dy, starts=starts, scale=0.7)
    torch.testing.assert_close(got["y"][inside], y.detach()[inside])
    for n, w in zip(("dq", "dk", "dv"), want):
        torch.testing.assert_close(got[n][inside], w[inside])
        assert torch.isnan(got[n][~inside]).all()
    assert (got["y_1"][inside] >= got["y"][inside].abs() - 1e-15).all()


def test_oracle_attention_closed_forms():
    gen = torch.Generator().manual_seed(2)
    v = rn(gen, 1, 6, 1, 4)
    zero = torch.zeros(1, 6, 1, 4, dtype=torch.float64)
    o = R.attention(zero, rn(gen, 1, 6, 1, 4), v)
    torch.testing.assert_close(o["y"], v.cumsum(1) / torch.arange(1, 7).view(1, 6, 1, 1))
    torch.testing.assert_close(o["lse"][0, :, 0], torch.log(torch.arange(1, 7).double()))
    # one key far ahead takes all of the weight
    k = zero.clone()
    k[0, 2, 0, 0] = 1e4
    q = zero + 1
    torch.testing.assert_close(R.attention(q, k, v)["y"][0, 2:], v[0, 2:3].expand(4, 1, 4))


def test_oracle_decode_is_the_prompt():
    """Over the cache the last tokens get what the whole sequence gets."""
    gen = torch.Generator().manual_seed(3)
    q, k, v = rn(gen, 1, 37, 4, 8), rn(gen, 1, 37, 2, 8), rn(gen, 1, 37, 2, 8)
    want = R.attention(q, k, v)["y"]
    pages = [torch.full((5, 2, 16, 8), 9.0, dtype=torch.float64) for _ in range(2)]
    table = [[4, 0, 2]]
    for i in range(37):
        for p, x in zip(pages, (k, v)):
            p[table[0][i // 16], :, i % 16] = x[0, i]
    got = R.decode(q[:, 34:], *pages, table, [37])["y"]
    torch.testing.assert_close(got, want[:, 34:])
    assert (R.decode(q[:, :1], *pages, table, [0])["y"] == 0).all()
    assert R.places([37], [2], table, 16, 5) == [[(2, 3), (2, 4)]]
    assert R.places([1], [3], table, 16, 5) == [[None, None, (4, 0)]]


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_qk_norm(interleaved):
    gen = torch.Generator().manual_seed(4)
    q, k, dq, dk = rn(gen, 2, 3, 2, 8), rn(gen, 2, 3, 1, 8), rn(gen, 2, 3, 2, 8), rn(gen, 2, 3, 1, 8)
    wq, wk, theta, pos = rn(gen, 8), rn(gen, 8), rn(gen, 2), torch.tensor([[0, 5, -3], [7, 7, 100]])
    a = [x.clone().requires_grad_() for x in (q, k, wq, wk)]
    out = []
    for x, w in ((a[0], a[2]), (a[1], a[3])):
        n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        c = torch.polar(torch.ones(()).double(), pos[..., None, None] * theta)
        z = torch.complex(n[..., 0:4:2], n[..., 1:4:2]) if interleaved else torch.complex(n[..., 0:2], n[..., 2:4])
        z = z * c
        turned = torch.stack((z.real, z.imag), -1).flatten(-2) if interleaved else torch.cat((z.real, z.imag), -1)
        out.append(torch.cat((turned, n[..., 4:]), -1))
    want = torch.autograd.grad((out[0] * dq).sum() + (out[1] * dk).sum(), a)
    got = R.qk_norm(q, k, wq, wk, theta, pos, dq, dk, interleaved=interleaved)
    torch.testing.assert_close(got["q"], out[0].detach())
    torch.testing.assert_close(got["k"], out[1].detach())
    for n, w in zip(("dq", "dk", "dwq", "dwk"), want):
        torch.testing.assert_close(got[n], w)


def test_oracle_e4m3():
    """Against torch's own conversion on the CPU, where that is in range."""
    gen = torch.Generator().manual_seed(5)
    x = torch.cat((torch.randn(20000, generator=gen) * 60, torch.randn(20000, generator=gen) * 0.01,
                   torch.tensor([0.0, 448.0, -448.0, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9])))
    x = x.clamp(-448, 448)
    assert torch.equal(R.e4m3(x), x.to(torch.float8_e4m3fn).double())
    assert R.e4m3(torch.tensor([1e9])) == 448
    z, s = R.quantise(torch.zeros(2, 4))
    assert (z == 0).all() and (s == 0).all()


# ------------------------------------------------------------------- the C ABI

def test_exports_every_declared_symbol():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "attention.h")).read(), flags=re.S)
    declared = set(re.findall(r"\b((?:attn|kv|qk_norm)_[a-z_0-9]+)\s*\(", src))
    assert declared == set(_lib.ATTENTION_EXPORTS)
    for n in _lib.ATTENTION_EXPORTS:
        assert hasattr(_lib.lib(), n), n
    for n in pkg.__all__:
        assert callable(getattr(pkg, n)), n


FAKE = 0x10000   # aligned, never dereferenced: the calls below end in validation


def attn_shape(B=2, T=70, Hq=4, Hk=2, D=64, nseq=0, q=0, k=0, v=0, dtype=1, flags=0, scale=0.125):
    return _lib.AttnShape(B, T, Hq, Hk, D, nseq, q, k, v, dtype, flags, scale)


BAD_ATTN = [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(Hq=3), INVALID), (dict(Hq=0), INVALID), (dict(Hk=0), INVALID),
    (dict(D=0), INVALID), (dict(nseq=-1), INVALID), (dict(nseq=2), INVALID), (dict(dtype=2), INVALID),
    (dict(flags=1), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=1e-40), INVALID), (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED),
    (dict(Hq=65538, Hk=2), UNSUPPORTED), (dict(B=1, T=2 ** 30 + 1), UNSUPPORTED), (dict(B=1, nseq=65536), UNSUPPORTED),
    (dict(q=255), INVALID), (dict(q=260), INVALID), (dict(k=64), INVALID), (dict(v=-8), INVALID), (dict(q=2 ** 22 + 8), UNSUPPORTED),
    (dict(B=2 ** 40, T=2 ** 30), INVALID), (dict(B=2 ** 20, T=2 ** 20), UNSUPPORTED),
    (dict(B=1, T=2 ** 30, Hq=8, Hk=8), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,want", BAD_ATTN, ids=[str(c[0]) for c in BAD_ATTN])
def test_attention_refuses_shapes(kw, want):
    L, sh = _lib.lib(), attn_shape(**kw)
    st = FAKE if kw.get("nseq", 0) > 0 else None
    r = ctypes.byref(sh)
    assert L.attn_forward(r, FAKE, FAKE, FAKE, st, FAKE, FAKE, None, None) == want
    assert L.attn_backward(r, FAKE, FAKE, FAKE, st, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 40, None) == want
    assert L.attn_record_bytes(r) == 0 and L.attn_backward_workspace_bytes(r) == 0


def test_attention_refuses_pointers():
    L = _lib.lib()
    fwd = dict(q=FAKE, k=FAKE, v=FAKE, starts=None, y=FAKE, lse=FAKE, rec=FAKE)
    bwd = dict(q=FAKE, k=FAKE, v=FAKE, starts=None, y=FAKE, lse=FAKE, rec=FAKE, dy=FAKE, dq=FAKE, dk=FAKE, dv=FAKE)
    sh = attn_shape()
    need = L.attn_backward_workspace_bytes(ctypes.byref(sh))
    assert need == -(-2 * 70 * 4 * 8 // 256) * 256 and L.attn_record_bytes(ctypes.byref(sh)) == 2 * 70 * 4 * 64 * 2

    def f(shape=sh, **kw):
        return L.attn_forward(ctypes.byref(shape), *{**fwd, **kw}.values(), None)

    def b(shape=sh, ws=FAKE, size=None, **kw):
        return L.attn_backward(ctypes.byref(shape), *{**bwd, **kw}.values(), ws, need if size is None else size, None)

    for n in ("q", "k", "v", "y"):
        assert f(**{n: None}) == INVALID and f(**{n: FAKE + 8}) == INVALID, n
    for n in bwd:
        if n not in ("starts", "rec"):
            assert b(**{n: None}) == INVALID, n
        assert b(**{n: FAKE + 2}) == INVALID, n
    assert f(lse=FAKE + 2) == INVALID and f(rec=FAKE + 8) == INVALID
    assert f(starts=FAKE) == INVALID and f(shape=attn_shape(B=1, nseq=3)) == INVALID
    assert f(shape=attn_shape(B=1, nseq=3), starts=FAKE + 2) == INVALID
    assert f(shape=attn_shape(dtype=0)) == INVALID          # a record with fp32 inputs
    assert b(shape=attn_shape(dtype=0)) == INVALID
    assert b(ws=None) == WORKSPACE and b(size=need - 1) == WORKSPACE and b(ws=FAKE + 16) == WORKSPACE
    assert L.attn_forward(None, *fwd.values(), None) == INVALID
    # nothing to do: nothing is needed
    for kw in (dict(B=0), dict(T=0), dict(Hq=0, Hk=0)):
        e = attn_shape(**kw)
        assert L.attn_forward(ctypes.byref(e), *[None] * 7, None) == OK
        assert L.attn_backward(ctypes.byref(e), *[None] * 11, None, 0, None) == OK


def qk_shape(B=2, T=5, Hq=4, Hk=2, D=64, R_=64, q=0, k=0, dtype=1, flags=0, eps=1e-6):
    return _lib.QkNormShape(B, T, Hq, Hk, D, R_, q, k, dtype, flags, eps)


BAD_QK = [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(Hq=-1), INVALID), (dict(D=0), INVALID), (dict(R_=-16), INVALID),
    (dict(R_=80), INVALID), (dict(R_=8), UNSUPPORTED), (dict(R_=40), UNSUPPORTED), (dict(D=32), UNSUPPORTED),
    (dict(Hk=70000), UNSUPPORTED), (dict(dtype=7), INVALID), (dict(flags=2), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(q=250), INVALID), (dict(k=4), INVALID), (dict(k=2 ** 23), UNSUPPORTED),
    (dict(B=2 ** 40, T=2 ** 40), INVALID),
]


@pytest.mark.parametrize("kw,want", BAD_QK, ids=[str(c[0]) for c in BAD_QK])
def test_qk_norm_refuses_shapes(kw, want):
    L, r = _lib.lib(), ctypes.byref(qk_shape(**kw))
    assert L.qk_norm_forward(r, *[FAKE] * 8, None) == want
    assert L.qk_norm_backward(r, *[FAKE] * 12, FAKE, 1 << 40, None) == want
    assert L.qk_norm_workspace_bytes(r) == 0


def test_qk_norm_refuses_pointers():
    L = _lib.lib()
    r = ctypes.byref(qk_shape())
    fwd = dict(q=FAKE, k=FAKE, wq=FAKE, wk=FAKE, theta=FAKE, pos=None, qz=FAKE, kz=FAKE)
    for bad in (dict(q=None), dict(k=None), dict(wq=None), dict(wk=None), dict(theta=None), dict(qz=None), dict(kz=None),
                dict(q=FAKE + 8), dict(wq=FAKE + 4), dict(theta=FAKE + 2), dict(pos=FAKE + 2), dict(kz=FAKE + 8)):
        assert L.qk_norm_forward(r, *{**fwd, **bad}.values(), None) == INVALID, bad
    bwd = dict(dqz=FAKE, dkz=FAKE, q=FAKE, k=FAKE, wq=FAKE, wk=FAKE, theta=FAKE, pos=None, dq=FAKE, dk=FAKE, dwq=FAKE, dwk=FAKE)
    need = L.qk_norm_workspace_bytes(r)
    assert need == 10 * 2 * 64 * 4
    for bad in (dict(dqz=None), dict(dkz=None), dict(q=None), dict(dq=None), dict(dwq=None), dict(dwk=None), dict(wq=None),
                dict(wq=None, wk=None), dict(dk=FAKE + 8), dict(theta=None)):
        assert L.qk_norm_backward(r, *{**bwd, **bad}.values(), FAKE, need, None) == INVALID, bad
    assert L.qk_norm_backward(r, *bwd.values(), FAKE, need - 1, None) == WORKSPACE
    assert L.qk_norm_backward(r, *bwd.values(), None, need, None) == WORKSPACE
    assert L.qk_norm_forward(ctypes.byref(qk_shape(R_=0)), *fwd.values(), None) == INVALID   # theta without entries that turn
    assert L.qk_norm_forward(ctypes.byref(qk_shape(T=0)), *[None] * 4, FAKE, None, None, None, None) == OK


def cache_shape(rows=3, T=4, Hk=2, D=64, packed=0, pages=9, page=16, most=4, k=0, v=0, dtype=1, kind=0):
    return _lib.KvCacheShape(rows, T, Hk, D, packed, pages, page, most, k, v, dtype, kind)


BAD_CACHE = [
    (dict(rows=-1), INVALID), (dict(T=-1), INVALID), (dict(Hk=-1), INVALID), (dict(D=0), INVALID), (dict(D=80), UNSUPPORTED),
    (dict(packed=2), INVALID), (dict(pages=-1), INVALID), (dict(pages=2 ** 31), UNSUPPORTED), (dict(page=0), INVALID),
    (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(page=512), UNSUPPORTED), (dict(most=-1), INVALID),
    (dict(most=2 ** 27), UNSUPPORTED), (dict(most=2 ** 62), INVALID), (dict(dtype=3), INVALID), (dict(kind=2), INVALID),
    (dict(k=100), INVALID), (dict(v=64), INVALID), (dict(Hk=70000), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,want", BAD_CACHE, ids=[str(c[0]) for c in BAD_CACHE])
def test_cache_refuses_shapes(kw, want):
    L, r = _lib.lib(), ctypes.byref(cache_shape(**kw))
    scales = [FAKE, FAKE] if kw.get("kind") else [None, None]
    st = FAKE if kw.get("packed") else None
    assert L.kv_write(r, FAKE, FAKE, FAKE, FAKE, *scales, FAKE, FAKE, st, None) == want
    if "k" not in kw and "v" not in kw:
        assert L.kv_read(r, FAKE, FAKE, *scales, FAKE, FAKE, st, FAKE, FAKE, None) == want


def test_cache_refuses_pointers():
    L = _lib.lib()
    a = dict(k=FAKE, v=FAKE, kp=FAKE, vp=FAKE, ks=None, vs=None, table=FAKE, lens=FAKE, starts=None)
    r = ctypes.byref(cache_shape())
    for bad in (dict(k=None), dict(v=None), dict(kp=None), dict(vp=None), dict(table=None), dict(lens=None), dict(ks=FAKE),
                dict(vs=FAKE), dict(starts=FAKE), dict(k=FAKE + 8), dict(kp=FAKE + 8), dict(table=FAKE + 2), dict(lens=FAKE + 1)):
        assert L.kv_write(r, *{**a, **bad}.values(), None) == INVALID, bad
    r8 = ctypes.byref(cache_shape(kind=1))
    assert L.kv_write(r8, *a.values(), None) == INVALID
    assert L.kv_write(r8, *{**a, "ks": FAKE, "vs": FAKE + 2}.values(), None) == INVALID
    assert L.kv_write(ctypes.byref(cache_shape(packed=1)), *a.values(), None) == INVALID
    assert L.kv_read(ctypes.byref(cache_shape(k=256)), FAKE, FAKE, None, None, FAKE, FAKE, None, FAKE, FAKE, None) == INVALID
    for kw in (dict(rows=0), dict(T=0), dict(Hk=0)):
        assert L.kv_write(ctypes.byref(cache_shape(**kw)), *[None] * 9, None) == OK
        assert L.kv_read(ctypes.byref(cache_shape(**kw)), *[None] * 9, None) == OK
    # a pool or a table of no pages: nothing is written
    assert L.kv_write(ctypes.byref(cache_shape(pages=0)), FAKE, FAKE, *[None] * 4, FAKE, FAKE, None, None) == OK
    assert L.kv_write(ctypes.byref(cache_shape(most=0)), FAKE, FAKE, FAKE, FAKE, None, None, None, FAKE, None, None) == OK


def decode_shape(B=2, T=1, Hq=8, Hk=2, D=128, pages=100, page=64, most=128, q=0, dtype=1, kind=0, scale=0.1):
    return _lib.AttnDecodeShape(B, T, Hq, Hk, D, pages, page, most, q, dtype, kind, scale)


BAD_DECODE = [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(Hq=7), INVALID), (dict(Hq=0), INVALID), (dict(D=32), UNSUPPORTED),
    (dict(B=65536), UNSUPPORTED), (dict(T=65536), UNSUPPORTED), (dict(Hq=64, Hk=1, T=65535), UNSUPPORTED), (dict(page=24), UNSUPPORTED),
    (dict(page=-16), INVALID), (dict(most=2 ** 26), UNSUPPORTED), (dict(q=8), INVALID), (dict(dtype=5), INVALID),
    (dict(kind=-1), INVALID), (dict(scale=-0.1), INVALID), (dict(scale=0.0), INVALID),
]


@pytest.mark.parametrize("kw,want", BAD_DECODE, ids=[str(c[0]) for c in BAD_DECODE])
def test_decode_refuses_shapes(kw, want):
    L, r = _lib.lib(), ctypes.byref(decode_shape(**kw))
    assert L.attn_decode(r, FAKE, FAKE, FAKE, None, None, FAKE, FAKE, FAKE, FAKE, 1 << 40, None) == want
    assert L.attn_decode_workspace_bytes(r) == 0


def test_decode_refuses_pointers():
    L = _lib.lib()
    a = dict(q=FAKE, kp=FAKE, vp=FAKE, ks=None, vs=None, table=FAKE, lens=FAKE, y=FAKE)
    r = ctypes.byref(decode_shape())
    need = L.attn_decode_workspace_bytes(r)
    assert need > 0 and need % 256 == 0
    for bad in (dict(q=None), dict(kp=None), dict(vp=None), dict(table=None), dict(lens=None), dict(y=None), dict(ks=FAKE),
                dict(q=FAKE + 8), dict(vp=FAKE + 4), dict(table=FAKE + 2), dict(y=FAKE + 8)):
        assert L.attn_decode(r, *{**a, **bad}.values(), FAKE, need, None) == INVALID, bad
    assert L.attn_decode(ctypes.byref(decode_shape(kind=1)), *a.values(), FAKE, need, None) == INVALID
    assert L.attn_decode(r, *a.values(), FAKE, need - 1, None) == WORKSPACE
    assert L.attn_decode(r, *a.values(), None, need, None) == WORKSPACE
    for kw in (dict(B=0), dict(T=0), dict(Hq=0, Hk=0)):
        e = ctypes.byref(decode_shape(**kw))
        assert L.attn_decode_workspace_bytes(e) == 0 and L.attn_decode(e, *[None] * 8, None, 0, None) == OK
    # one step is one part
    assert L.attn_decode_workspace_bytes(ctypes.byref(decode_shape(most=1, page=16))) == 0


# ------------------------------------------------------------- the binding

def test_binding_refuses():
    q, k = torch.zeros(2, 3, 4, 64), torch.zeros(2, 3, 2, 64)
    with pytest.raises(ValueError, match="device tensor"):
        api.attn_forward(q, k, k)
    with pytest.raises(ValueError, match="dtype"):
        api.attn_forward(q.half(), k.half(), k.half())
    with pytest.raises(ValueError, match="Hq"):
        api.qk_norm_forward(q[0], k[0])
    with pytest.raises(ValueError):
        api.kv_write(k, k, k, k, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        api.kv_read(k, k, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), T=1)
    with pytest.raises(ValueError):
        api.attn_decode(q, k, k, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


def test_binding_sizes():
    assert pkg.attn_record_bytes(2, 70, 4, 2, 64) == 2 * 70 * 4 * 64 * 2
    assert pkg.attn_record_bytes(2, 70, 4, 2, 64, torch.float32) == 0
    assert pkg.attn_backward_workspace_bytes(2, 70, 4, 2, 64) == -(-2 * 70 * 4 * 8 // 256) * 256
    assert pkg.qk_norm_workspace_bytes(2, 5, 4, 2, 64) == 10 * 2 * 64 * 4
    assert pkg.attn_decode_workspace_bytes(2, 1, 8, 2, 128, 100, 64, 128) > 0
    # a head size that the library does not take
    assert pkg.attn_record_bytes(2, 70, 4, 2, 0) == 0 and pkg.attn_backward_workspace_bytes(2, 70, 4, 2, 80) == 0


def test_unsupported_names_the_header():
    assert "attention.h" in _lib.status_text(UNSUPPORTED)
