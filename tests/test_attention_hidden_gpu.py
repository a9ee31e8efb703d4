"""Values that a token does not see, on the device: infinities and NaN there
reach nothing, and where they are seen they reach what the formulas say,
MI355X only.

A hidden value has weight 0, and 0 times any finite value is 0, so that a result
which does not see the value has the same bits as with a finite one in its place:
no tolerance is needed.  (dk and dv of the tile that the value lies in are summed in
another order then, and are compared with the oracle.)"""
import math

import pytest
import torch

import oracle.attention as R
from linear_attention_rnn_wkv7_amd import api
from test_attention_gpu import cache, cargs, check

pytestmark = pytest.mark.gpu
F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn


def randn(gen, *s):
    return torch.randn(s, generator=gen)


SHAPES = [
    # B, T, Hq, Hk, D, dtype, starts: few workgroups (the narrow form) and many (the wide one)
    (1, 100, 2, 1, 64, BF16, None), (2, 75, 2, 2, 128, BF16, None), (1, 90, 4, 2, 64, F32, None), (1, 70, 2, 1, 128, F32, None),
    (1, 300, 4, 2, 64, BF16, [0, 3, 3, 101, 290]),
    (9, 233, 16, 16, 64, BF16, None), (9, 233, 32, 16, 128, BF16, None), (17, 161, 16, 16, 64, F32, None),
    (9, 150, 32, 32, 128, F32, None), (1, 3000, 16, 8, 64, BF16, [0, 40] + [41 + 59 * i for i in range(51)]),
]
IDS = ["-".join(map(str, c[:6])).replace("torch.", "") + ("-packed" if c[6] else "") for c in SHAPES]


def inputs(case, seed):
    B, T, Hq, Hk, D, dt, starts = case
    gen = torch.Generator().manual_seed(seed)
    d = {n: (randn(gen, B, T, h, D)).to(dt).cuda() for n, h in (("q", Hq), ("k", Hk), ("v", Hk), ("dy", Hq))}
    return d, None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")


def places(case):
    """(row, token, sequence's first token and end) in some sequences of the case."""
    B, T, starts = case[0], case[1], case[6]
    if starts is None:
        at = [0, 1, 30, 31, 32, 33, 63, 64, 66, 95, 127, 128, 140, 160, T - 2, T - 1]
        return [(i % B, t, 0, T) for i, t in enumerate(t for t in at if t < T)]
    out = []
    for lo, hi in list(zip(starts[:-1], starts[1:]))[-8:]:
        out += [(0, t, lo, hi) for t in (lo, lo + 17, lo + 33, hi - 1) if lo <= t < hi]
    return out


def inside(case):
    m = torch.zeros(case[0], case[1], dtype=torch.bool, device="cuda")
    if case[6] is None:
        return ~m
    m[:, case[6][0]:case[6][-1]] = True
    return m


def same(a, b, keep, label):
    """a and b are bit for bit the same where keep holds."""
    x, y = (t.contiguous().view(torch.int32 if t.dtype is F32 else torch.int16) for t in (a, b))
    assert (x == y)[keep].all(), label


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("case", SHAPES, ids=IDS)
def test_forward_values(case, bad):
    """One entry of one token's v: it reaches that entry of the tokens from there on."""
    B, T, Hq, Hk, D, dt, _ = case
    d, st = inputs(case, 1)
    args = d["q"], d["k"]
    clean, lse, rec = api.attn_forward(*args, d["v"], seq_starts=st, want_lse=True, want_record=True)
    for n, (b, t, lo, hi) in enumerate(places(case)):
        v, g, e = d["v"].clone(), n % Hk, (7 * n + 5) % D
        v[b, t, g, e] = bad
        y, lse2, rec2 = api.attn_forward(*args, v, seq_starts=st, want_lse=True, want_record=True)
        heads = slice(g * (Hq // Hk), (g + 1) * (Hq // Hk))
        keep = inside(case)[:, :, None, None].expand_as(y).clone()
        keep[b, t:hi, heads, e] = False
        same(y, clean, keep, (case, b, t))
        if rec is not None:
            same(rec2, rec, keep, (case, b, t))
        same(lse2, lse, keep[..., (e + 1) % D], (case, b, t))
        hit = y[b, t:hi, heads, e]
        assert (torch.isnan(hit) if math.isnan(bad) else hit == bad).all(), (case, b, t)


def backward(d, starts):
    a = d["q"], d["k"], d["v"]
    y, lse, rec = api.attn_forward(*a, seq_starts=starts, want_lse=True, want_record=True)
    return api.attn_backward(*a, y, lse, d["dy"], rec, seq_starts=starts)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("case", SHAPES, ids=IDS)
def test_dq(case, bad):
    """One entry of one token's k, or of its v: dq of the tokens before it, of other
    sequences and of other heads does not notice; from there on it is seen."""
    B, T, Hq, Hk, D, dt, _ = case
    d, st = inputs(case, 2)
    clean = backward(d, st)["dq"]
    for n, (b, t, lo, hi) in enumerate(places(case)):
        for name in ("k", "v"):
            x, g, e = d[name].clone(), n % Hk, (7 * n + 5) % D
            x[b, t, g, e] = bad
            dq = backward({**d, name: x}, st)["dq"]
            heads = slice(g * (Hq // Hk), (g + 1) * (Hq // Hk))
            keep = inside(case)[:, :, None, None].expand_as(dq).clone()
            keep[b, t:hi, heads] = False
            same(dq, clean, keep, (case, name, b, t))
            assert not torch.isfinite(dq[b, t:hi, heads, e]).any(), (case, name, b, t)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("case", SHAPES, ids=IDS)
def test_dk_dv(case, bad):
    """One entry of one token's dy, or of its q: the keys behind it, of other sequences
    and of other heads do not notice.  In dv the entry of a dy is seen as it is, by
    itself; nothing of dk is finite then."""
    B, T, Hq, Hk, D, dt, starts = case
    d, st = inputs(case, 3)
    if starts is not None:
        for n in d:
            d[n][:, ~inside(case)[0]] = 0
    clean = backward(d, st)
    exact = R.attention(d["q"], d["k"], d["v"], d["dy"], starts=starts)
    longest = T if starts is None else max(b - a for a, b in zip(starts[:-1], starts[1:]))
    for n, (b, t, lo, hi) in enumerate(places(case)):
        for name in ("dy", "q"):
            x, h, e = d[name].clone(), (5 * n + 1) % Hq, (7 * n + 5) % D
            g = h * Hk // Hq
            x[b, t, h, e] = bad
            got = backward({**d, name: x}, st)
            label = (case, name, b, t)
            keep = inside(case)[:, :, None, None].expand_as(got["dk"]).clone()
            keep[b, lo:hi, g] = False
            for m in ("dk", "dv"):
                same(got[m], clean[m], keep, label)
            keep = inside(case)[:, :, None, None].expand_as(got["dq"]).clone()
            keep[b, t, h] = False
            same(got["dq"], clean["dq"], keep, label)
            behind = slice(t + 1, hi)
            want = {m: w[b:b + 1, behind, g:g + 1] for m, w in exact.items() if m[:2] in ("dk", "dv")}
            check({m: got[m][b:b + 1, behind, g:g + 1] for m in ("dk", "dv")}, want, str(label), D=D, T=longest)
            seen = got["dv"][b, lo:t + 1, g]
            if name == "dy":
                assert (torch.isnan(seen[:, e]) if math.isnan(bad) else seen[:, e] == bad).all(), label
                assert not torch.isfinite(got["dk"][b, lo:t + 1, g]).any(), label
                want = {m: w[b:b + 1, lo:t + 1, g:g + 1].clone() for m, w in exact.items() if m[:2] == "dv"}
                want["dv"][..., e] = math.nan   # not compared
                check({"dv": got["dv"][b:b + 1, lo:t + 1, g:g + 1]}, want, str(label), D=D, T=longest)
            else:
                assert not torch.isfinite(got["dk"][b, lo:t + 1, g, e]).any(), label


@pytest.mark.parametrize("dt, B, H", [(BF16, 1, 2), (F32, 1, 2), (BF16, 130, 2), (F32, 130, 4)])
def test_rows_behind_the_last(dt, B, H):
    """A length that ends inside a tile, a key whose scores are all minus infinity and an
    infinity in the last dy: what stands for the rows behind the last adds nothing."""
    d, _ = inputs((B, 77, H, H, 64, dt, None), 4)
    d["q"].abs_().add_(0.1)
    d["k"][:, 40] = -math.inf
    clean = backward(d, None)
    assert torch.isfinite(clean["dk"]).all() and torch.isfinite(clean["dv"]).all()
    assert (clean["dk"][:, 40] == 0).all() and (clean["dv"][:, 40] == 0).all()
    dy = d["dy"].clone()
    dy[:, -1, :, 3] = math.inf
    dv = backward({**d, "dy": dy}, None)["dv"]
    others = torch.arange(64, device="cuda") != 3
    assert (dv[:, torch.arange(77) != 40, :, 3] == math.inf).all()
    assert (dv[:, 40][..., others] == 0).all() and torch.isfinite(dv[..., others]).all()


DECODE = [
    # B, T, Hq, Hk, D, page, most, dtype, kind, lens
    (2, 2, 4, 2, 64, 16, 5, BF16, BF16, [80, 33]), (2, 5, 12, 2, 128, 32, 9, BF16, BF16, [287, 4]),
    (2, 3, 6, 2, 64, 64, 4, F32, F32, [200, 65]), (1, 4, 2, 1, 128, 16, 60, F32, F32, [932]),
    (2, 4, 32, 8, 64, 128, 3, BF16, E4M3, [383, 130]), (1, 6, 40, 1, 128, 256, 2, BF16, E4M3, [512]),
    (2, 5, 3, 3, 64, 16, 8, F32, E4M3, [100, 35]), (1, 70, 6, 2, 64, 16, 20, BF16, BF16, [311]),
    (1, 70, 6, 2, 128, 16, 20, BF16, E4M3, [311]), (2, 40, 4, 4, 64, 32, 4, F32, F32, [70, 20]),
]


@pytest.mark.parametrize("case", DECODE, ids=["-".join(map(str, c[:9])).replace("torch.", "") for c in DECODE])
def test_decode_values(case):
    """One entry of a new token's v in the cache (or its scale): the tokens before it do
    not notice, the others see it."""
    B, T, Hq, Hk, D, page, most, dt, kind, lens = case
    c = cache(B, most, page, Hk, D, dt, kind, seed=90)
    gen = torch.Generator().manual_seed(91)
    q = randn(gen, B, T, Hq, D).to(dt).cuda()
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    clean = api.attn_decode(q, *cargs(c, ln))
    last = [(b, n - 1 - i) for b, n in enumerate(lens) for i in {0, 1, T // 2, T - 1, T, T + 40} if i < n]
    for m, (b, pos) in enumerate(last):
        place, at, g, e = int(c["table"][b, pos // page]), pos % page, m % Hk, (7 * m + 5) % D
        heads = slice(g * (Hq // Hk), (g + 1) * (Hq // Hk))
        t = max(0, pos - (lens[b] - T))      # the first token that sees it
        for bad in ("nan", "inf", "scale"):
            if (bad == "scale") != (kind is E4M3) and bad != "nan":
                continue
            x = {n: y if y is None or n == "table" else y.clone() for n, y in c.items()}
            if bad == "scale":
                x["v_scale"][place, g, at] = math.nan
            elif kind is E4M3:
                x["v_pages"].view(torch.uint8)[place, g, at, e] = 0xFF
            else:
                x["v_pages"][place, g, at, e] = math.nan if bad == "nan" else -math.inf
            y = api.attn_decode(q, *cargs(x, ln))
            keep = torch.ones_like(y, dtype=torch.bool)
            keep[b, t:, heads, slice(None) if bad == "scale" else e] = False
            same(y, clean, keep, (case, b, pos, bad))
            hit = y[~keep]
            # (an infinity times the second part of a weight in two, which may be 0 or below, is any of them)
            want = ~torch.isfinite(hit) if bad == "inf" and dt is BF16 else hit == -math.inf if bad == "inf" else torch.isnan(hit)
            assert want.all(), (case, b, pos, bad)
