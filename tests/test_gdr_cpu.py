"""The gated delta rule, its epilogue and the residual norm without a GPU:
the oracle against autograd, differences and closed forms; the C ABI's
exports, sizes and refusals (no call here launches a kernel)."""
import ctypes
import os
import re

import pytest
import torch

import oracle.gdr as R
from linear_attention_rnn_wkv7_amd import _lib, api

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, WORKSPACE = _lib.WKV7_ERR_INVALID, _lib.WKV7_ERR_UNSUPPORTED, _lib.WKV7_ERR_WORKSPACE


# ------------------------------------------------------------------ the oracle

def _inputs(seed, B, T, Hk, Hv, K, V, seqs):
    gen = torch.Generator().manual_seed(seed)

    def rn(*s):
        return torch.randn(s, generator=gen, dtype=torch.float64)

    return dict(q=rn(B, T, Hk, K), k=rn(B, T, Hk, K) / K ** 0.5, v=rn(B, T, Hv, V),
                g=-rn(B, T, Hv).abs(), beta=torch.sigmoid(rn(B, T, Hv)), s0=rn(seqs, Hv, V, K),
                dy=rn(B, T, Hv, V), dsT=rn(seqs, Hv, V, K))


def _loss(d, starts, norm):
    """The definition in differentiable torch, as matrices."""
    B, T, Hk, K = d["q"].shape
    Hv = d["v"].shape[2]
    seqs = [(b, 0, T) for b in range(B)] if starts is None else [(0, *p) for p in zip(starts, starts[1:])]
    total = 0
    for i, (b, lo, hi) in enumerate(seqs):
        for h in range(Hv):
            S = d["s0"][i, h]
            for t in range(lo, hi):
                q, k = d["q"][b, t, h * Hk // Hv], d["k"][b, t, h * Hk // Hv]
                if norm:
                    q, k = (x / torch.sqrt(x @ x + 1e-6) for x in (q, k))
                be = d["beta"][b, t, h]
                S = torch.exp(d["g"][b, t, h]) * S @ (torch.eye(K, dtype=S.dtype) - be * torch.outer(k, k))
                S = S + be * torch.outer(d["v"][b, t, h], k)
                total = total + (S @ q) @ d["dy"][b, t, h] * K ** -0.5
            total = total + (S * d["dsT"][i, h]).sum()
    return total


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("starts", [None, [0, 0, 1, 5, 7]])
def test_oracle_rule_gradients(starts, norm):
    B, T, seqs = (2, 5, 2) if starts is None else (1, 7, 4)
    d = _inputs(3, B, T, 2, 4, 3, 2, seqs)
    names = ("q", "k", "v", "g", "beta", "s0")
    leaves = {n: d[n].clone().requires_grad_() for n in names}
    loss = _loss({**d, **leaves}, starts, norm)
    grads = dict(zip(names, torch.autograd.grad(loss, [leaves[n] for n in names])))
    got = R.rule(*(d[n] for n in names), d["dy"], d["dsT"], starts=starts, norm_qk=norm)
    want = (got["y"] * d["dy"]).sum() + (got["sT"] * d["dsT"]).sum()
    assert abs(want - loss.detach()) <= 1e-12 * abs(want) + 1e-12
    for n in names:
        torch.testing.assert_close(got["d" + n], grads[n], rtol=1e-11, atol=1e-12)
    # differences of the oracle's own forward along one direction per input
    for n in names:
        gen = torch.Generator().manual_seed(9)
        e = torch.randn(d[n].shape, generator=gen, dtype=torch.float64)

        def value(s):
            o = R.rule(*({**d, n: d[n] + s * e}[m] for m in names), starts=starts, norm_qk=norm)
            return (o["y"] * d["dy"]).sum() + (o["sT"] * d["dsT"]).sum()

        diff = (value(1e-5) - value(-1e-5)) / 2e-5
        assert abs(diff - (got["d" + n] * e).sum()) <= 1e-6 * (1 + abs(diff)), n


def test_oracle_rule_closed_forms():
    # beta = 0 writes nothing: the state only decays
    d = _inputs(5, 1, 4, 1, 1, 3, 2, 1)
    o = R.rule(d["q"], d["k"], d["v"], d["g"], torch.zeros_like(d["beta"]), d["s0"], scale=1.0)
    torch.testing.assert_close(o["sT"][0, 0], torch.exp(d["g"].sum()) * d["s0"][0, 0])
    # a unit key with beta = 1 stores its value exactly
    k = torch.zeros(1, 1, 1, 3, dtype=torch.float64)
    k[..., 1] = 1
    o = R.rule(k, k, d["v"][:, :1], d["g"][:, :1], torch.ones(1, 1, 1), d["s0"], scale=1.0)
    torch.testing.assert_close(o["y"], d["v"][:, :1])


def test_oracle_norm_gradients():
    gen = torch.Generator().manual_seed(4)
    y, g, dz = (torch.randn(2, 3, 4, 8, generator=gen, dtype=torch.float64) for _ in range(3))
    for heads in (1, 4):
        w = torch.randn(heads, 8, generator=gen, dtype=torch.float64)
        a = [x.clone().requires_grad_() for x in (y, g, w)]
        z = a[0] / torch.sqrt((a[0] ** 2).mean(-1, keepdim=True) + 1e-6) * a[2] * torch.nn.functional.silu(a[1])
        o = R.epilogue(y, g, w, dz)
        torch.testing.assert_close(o["z"], z.detach())
        for n, x in zip(("dy", "dgate", "dw"), torch.autograd.grad(z, a, dz)):
            torch.testing.assert_close(o[n], x)
    x, y, dh, dx = (torch.randn(5, 7, generator=gen, dtype=torch.float64) for _ in range(4))
    w, s = (torch.randn(7, generator=gen, dtype=torch.float64) for _ in range(2))
    a = [t.clone().requires_grad_() for t in (x, y, w, s)]
    xo = a[0] + a[3] * a[1]
    h = xo / torch.sqrt((xo ** 2).mean(-1, keepdim=True) + 1e-6) * a[2]
    want = torch.autograd.grad((h * dh).sum() + (xo * dx).sum(), a)
    o = R.residual_norm(x, y, w, s)
    torch.testing.assert_close(o["h"], h.detach())
    b = R.residual_norm_backward(dh, dx, o["x_out"], w, y, s)
    for n, t in zip(("dx", "dy", "dw", "dscale"), want):
        torch.testing.assert_close(b[n], t)


# ------------------------------------------------------------------- the C ABI

def _declared(name, prefix):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", name)).read(), flags=re.S)
    return set(re.findall(r"\b(" + prefix + r"_[a-z_0-9]+)\s*\(", src))


def test_exports_every_declared_symbol():
    L = _lib.lib()
    for header, prefix, names in (("gdr.h", "gdr", _lib.GDR_EXPORTS),
                                  ("residual_norm.h", "residual_norm", _lib.RESIDUAL_NORM_EXPORTS)):
        assert _declared(header, prefix) == set(names)
        for n in names:
            assert hasattr(L, n), n


FAKE = 0x10000   # aligned, never dereferenced: the calls below end in validation


def _rule_shape(B=2, T=70, Hk=2, Hv=4, K=64, V=32, nseq=0, dtype=0, flags=0, scale=0.125):
    return _lib.GdrShape(B, T, Hk, Hv, K, V, nseq, dtype, flags, scale)


BAD_SHAPES = [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(Hk=-1), INVALID), (dict(K=0), INVALID),
    (dict(V=-16), INVALID), (dict(nseq=-1), INVALID), (dict(dtype=2), INVALID), (dict(flags=2), INVALID),
    (dict(Hk=3), INVALID), (dict(Hk=0), INVALID), (dict(nseq=2), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(K=32), UNSUPPORTED), (dict(K=256), UNSUPPORTED), (dict(V=24), UNSUPPORTED), (dict(V=272), UNSUPPORTED),
    (dict(Hk=70000, Hv=70000), UNSUPPORTED), (dict(B=70000), UNSUPPORTED),
    (dict(B=1 << 40, T=1 << 40), UNSUPPORTED), (dict(T=1 << 60), INVALID),
    (dict(B=1, T=1 << 32, nseq=1), INVALID),
]


def _forward(sh, ptrs=None, starts=None, outs=(FAKE, FAKE, None), ws=FAKE, ws_bytes=1 << 40):
    p = [FAKE] * 5 if ptrs is None else ptrs
    return _lib.lib().gdr_forward(ctypes.byref(sh) if sh is not None else None, *p, None, starts, *outs, ws,
                                  ws_bytes, None)


def _backward(sh, ptrs=None, starts=None, ws=FAKE, ws_bytes=1 << 40, outs=None):
    p = [FAKE] * 5 if ptrs is None else ptrs
    o = [FAKE] * 6 if outs is None else outs
    return _lib.lib().gdr_backward(ctypes.byref(sh), *p, None, starts, FAKE, None, None, *o, ws, ws_bytes, None)


def _decode(sh, pool=8, slots=FAKE, state=FAKE, y=FAKE, q=FAKE):
    return _lib.lib().gdr_decode(ctypes.byref(sh), q, FAKE, FAKE, FAKE, FAKE, state, pool, slots, y, None)


@pytest.mark.parametrize("change,want", BAD_SHAPES, ids=[str(c) for c, _ in BAD_SHAPES])
def test_rule_refuses_shapes(change, want):
    sh = _rule_shape(**change)
    starts = FAKE if sh.nseq > 0 else None
    assert _forward(sh, starts=starts) == want
    assert _backward(sh, starts=starts) == want
    if sh.nseq == 0:
        assert _decode(sh) == want
    L = _lib.lib()
    assert L.gdr_checkpoint_bytes(ctypes.byref(sh)) == 0
    assert L.gdr_forward_workspace_bytes(ctypes.byref(sh)) == 0
    assert L.gdr_backward_workspace_bytes(ctypes.byref(sh), 0) == 0


def test_rule_refuses_pointers():
    sh, packed = _rule_shape(), _rule_shape(B=1, nseq=3)
    assert _forward(None) == INVALID
    for i in range(5):
        for bad in (None, FAKE + 4):
            p = [FAKE] * 5
            p[i] = bad
            assert _forward(sh, p) == INVALID
            assert _backward(sh, p) == INVALID
    for i in range(3):
        outs = [None] * 3
        outs[i] = FAKE + 8
        assert _forward(sh, outs=outs) == INVALID
    for i in range(6):
        outs = [FAKE] * 6
        outs[i] = FAKE + 8
        assert _backward(sh, outs=outs) == INVALID
        if i < 5:
            outs[i] = None
            assert _backward(sh, outs=outs) == INVALID
    # the starts belong to packed shapes, and only to them
    for f in (_forward, _backward):
        assert f(sh, starts=FAKE) == INVALID
        assert f(packed, starts=None) == INVALID
        assert f(packed, starts=FAKE + 4) == INVALID
    assert _decode(packed) == INVALID
    assert _decode(sh, pool=-1) == INVALID
    assert _decode(sh, pool=1, slots=None) == INVALID      # two rows, one state
    assert _decode(sh, pool=1 << 31) == INVALID
    assert _decode(sh, state=None) == INVALID
    assert _decode(sh, y=None) == INVALID
    assert _decode(sh, q=FAKE + 2) == INVALID
    assert _decode(sh, slots=FAKE + 4) == INVALID


def test_rule_workspace():
    L = _lib.lib()
    sh = _rule_shape()
    back = L.gdr_backward_workspace_bytes(ctypes.byref(sh), 1)
    record = L.gdr_checkpoint_bytes(ctypes.byref(sh))
    assert back > record > 0
    assert L.gdr_backward_workspace_bytes(ctypes.byref(sh), 0) == back + record
    for ws, n in ((None, back + record), (FAKE, back), (FAKE + 16, back + record)):
        assert _backward(sh, ws=ws, ws_bytes=n) == WORKSPACE   # no record given
    # 2 rows of 2 chunks x 4 heads; packed: floor(70 / 64) + 3 chunks
    assert record == 2 * 2 * 4 * (64 * 32 + 64 * 32) * 4
    assert api.gdr_checkpoint_bytes(1, 70, 2, 4, 64, 32, nseq=3) == 4 * 4 * (64 * 32 + 64 * 32) * 4


def test_rule_without_work():
    """Empty batches, heads and pools return before any launch."""
    for change in (dict(B=0), dict(Hk=0, Hv=0)):
        sh = _rule_shape(**change)
        assert _forward(sh, [None] * 5, outs=(None, None, None), ws=None, ws_bytes=0) == 0
        assert _backward(sh, [None] * 5, ws=None, ws_bytes=0, outs=[None] * 6) == 0
        assert _decode(sh) == 0
    sh = _rule_shape(T=0)   # nothing asked for but y, which has no rows
    assert _forward(sh, [None] * 5, outs=(None, None, None), ws=None, ws_bytes=0) == 0
    assert _decode(sh) == 0
    assert _decode(_rule_shape(), pool=0) == 0


def test_epilogue_refusals():
    L = _lib.lib()

    def shape(rows=3, H=4, N=64, Hw=1, dtype=0, flags=0, eps=1e-6):
        return _lib.GdrEpilogueShape(rows, H, N, Hw, dtype, flags, eps)

    def fwd(sh, p=(FAKE,) * 4):
        return L.gdr_epilogue_forward(ctypes.byref(sh), *p, None)

    def bwd(sh, p=(FAKE,) * 7, ws=FAKE, n=1 << 40):
        return L.gdr_epilogue_backward(ctypes.byref(sh), *p, ws, n, None)

    for change, want in ((dict(rows=-1), INVALID), (dict(H=-1), INVALID), (dict(N=0), INVALID),
                         (dict(Hw=2), INVALID), (dict(Hw=0), INVALID), (dict(dtype=3), INVALID),
                         (dict(flags=1), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
                         (dict(N=8), UNSUPPORTED), (dict(N=48), UNSUPPORTED), (dict(N=512), UNSUPPORTED),
                         (dict(H=70000, Hw=70000), UNSUPPORTED), (dict(rows=1 << 40), UNSUPPORTED),
                         (dict(rows=1 << 62), INVALID)):
        assert fwd(shape(**change)) == want and bwd(shape(**change)) == want, change
    for i in range(4):
        for bad in (None, FAKE + 4):
            p = [FAKE] * 4
            p[i] = bad
            assert fwd(shape(), p) == INVALID
    for i in range(7):
        for bad in (None, FAKE + 4):
            p = [FAKE] * 7
            p[i] = bad
            assert bwd(shape(), p) == INVALID
    need = L.gdr_epilogue_workspace_bytes(ctypes.byref(shape()))
    assert need > 0
    for ws, n in ((None, need), (FAKE, need - 1), (FAKE + 16, need)):
        assert bwd(shape(), ws=ws, n=n) == WORKSPACE
    assert fwd(shape(rows=0), (None,) * 4) == 0
    assert fwd(shape(H=0, Hw=0), (None,) * 4) == 0 and bwd(shape(H=0, Hw=0), (None,) * 7, None, 0) == 0


def test_residual_norm_refusals():
    L = _lib.lib()

    def shape(rows=3, D=100, dtype=0, flags=0, eps=1e-6):
        return _lib.ResidualNormShape(rows, D, dtype, flags, eps)

    def fwd(sh, x=FAKE, y=FAKE, scale=FAKE, w=FAKE, xo=FAKE, h=FAKE):
        return L.residual_norm_forward(ctypes.byref(sh), x, y, scale, w, xo, h, None)

    def bwd(sh, dh=FAKE, dxo=FAKE, xo=FAKE, y=FAKE, scale=FAKE, w=FAKE, dx=FAKE, dy=FAKE, dw=FAKE, ds=FAKE,
            ws=FAKE, n=1 << 40):
        return L.residual_norm_backward(ctypes.byref(sh), dh, dxo, xo, y, scale, w, dx, dy, dw, ds, ws, n, None)

    for change, want in ((dict(rows=-1), INVALID), (dict(D=0), INVALID), (dict(dtype=2), INVALID),
                         (dict(flags=4), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("inf")), INVALID),
                         (dict(D=16385), UNSUPPORTED), (dict(rows=1 << 40), UNSUPPORTED)):
        assert fwd(shape(**change)) == want and bwd(shape(**change)) == want, change
    for n in ("x", "w", "h"):
        assert fwd(shape(), **{n: None}) == INVALID
    assert fwd(shape(), y=None) == INVALID          # a scale of nothing
    for n in ("x", "y", "scale", "w", "xo", "h"):
        assert fwd(shape(), **{n: FAKE + 4}) == INVALID
    for n in ("dh", "xo", "w", "dx", "dw", "y", "dy", "ds", "scale"):   # the last four come together
        assert bwd(shape(), **{n: None}) == INVALID, n
    for n in ("dh", "dxo", "xo", "y", "scale", "w", "dx", "dy", "dw", "ds"):
        assert bwd(shape(), **{n: FAKE + 4}) == INVALID
    need = L.residual_norm_workspace_bytes(ctypes.byref(shape()))
    for ws, n in ((None, need), (FAKE, need - 1), (FAKE + 16, need)):
        assert bwd(shape(), ws=ws, n=n) == WORKSPACE
    assert fwd(shape(rows=0), x=None, h=None) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 3, 2, 64)
    g = torch.zeros(1, 3, 2)
    with pytest.raises(ValueError):
        api.gdr_forward(x, x, x, g, g)
    with pytest.raises(ValueError):
        api.gdr_epilogue_forward(x, x, torch.ones(1, 64))
    with pytest.raises(ValueError):
        api.residual_norm_forward(x, x, torch.ones(64))
    with pytest.raises(ValueError):
        api.gdr_decode(x, x, x, g, g, torch.zeros(1, 2, 64, 64))


@pytest.mark.parametrize("change,want", [
    (dict(scale=1e-40), INVALID), (dict(scale=-1e-45), INVALID),     # denormal
    (dict(B=128, T=64 * 1024, Hk=33, Hv=33), UNSUPPORTED),           # 2^17 chunks x 33 heads
    (dict(B=1, T=64 * 65536, Hk=1, Hv=65, nseq=1), UNSUPPORTED)])    # 65537 slots x 65 heads
def test_rule_refuses_more_shapes(change, want):
    test_rule_refuses_shapes(change, want)


def test_rule_sizes_of_the_largest():
    """2^22 chunks times heads, and one fewer chunk's worth of heads than refused above."""
    sh = _rule_shape(B=128, T=64 * 1024, Hk=32, Hv=32, K=128, V=256)
    per = 128 * 1024 * 32
    assert _lib.lib().gdr_checkpoint_bytes(ctypes.byref(sh)) == per * 4 * (128 * 256 + 64 * 256)
    assert _lib.lib().gdr_backward_workspace_bytes(ctypes.byref(sh), 0) > 2 * per * 4 * (128 * 256 + 64 * 256)
