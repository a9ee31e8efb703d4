"""Softmax attention, the norm and rotation before it and the paged cache on
the device against the fp64 oracle (oracle.attention), MI355X only.

Bars.  fp32: a result passes through a score (a sum of D products), the
softmax's sum and a weighted sum (T terms each), the gradients through twice as
many.  Rounding errors of a sum add up like a random walk, sqrt(n) steps of
2^-24 of its size, those of a score become errors of a weight relative to it, and
twice that covers the exponential's own: F32 = 2 * 6 * sqrt(max(D, T)) * 2^-24
of the root mean square of the terms' sizes x_1, 16 times that for a single element.
dS = P (dy . v - D) is a difference of two sums of D products, each off by up to
F32 times |dy| . |v| (y is a mean of v: for D, |dy| . y_1), however small the
difference is: with a single key it is 0, and what is left are the two errors.
So dq and dk are also allowed 2 F32 x_d1.

bf16: one rounding of half a step, 2^-8, of the result and one of each weight:
at most 2^-8 (|x| + x_1) for an element, on top of the bar of fp32.  Roundings are
spread evenly over the step, with a third of the half step's square for a
variance, so that the 2-norm of the error is 2^-8 sqrt((|x|^2 + |x_2|^2) / 3),
taken 1.5 times.  D = dy . y takes y as the forward formed it: off by its weights'
roundings, at most 2^-8 y_1 (and 2^-8 y_2 / sqrt(3) on average), and by what the
record's rounding leaves, 2^-16 |y| (without a record, y's own 2^-8 |y|).  These
enter dq and dk as x_d1, x_d2 and x_d."""
import math

import pytest
import torch

import oracle.attention as R
from linear_attention_rnn_wkv7_amd import api

pytestmark = pytest.mark.gpu
F32, BF16, E4M3 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
HALF_STEP = {F32: 0.0, BF16: 2.0 ** -8}


def check(got, want, label, *, D, T, record=True, names=("y", "lse", "dq", "dk", "dv")):
    bar = 2 * 6 * max(D, T) ** 0.5 * 2.0 ** -24
    for n in names:
        if got.get(n) is None or n not in want:
            continue
        g, w = got[n].detach().cpu().double(), want[n]
        assert g.shape == w.shape, (label, n, g.shape, w.shape)
        keep = ~torch.isnan(w)
        g, w = g[keep], w[keep]
        if w.numel() == 0:
            continue
        assert torch.isfinite(g).all(), f"{label}: {n} is not finite"
        half = HALF_STEP[got[n].dtype]
        size = want[n + "_1"][keep] if n + "_1" in want else w.abs() + 1
        rms = float(size.norm()) / size.numel() ** 0.5
        extra = cancelled = 0.0
        if n + "_d1" in want:
            extra = cancelled = 2 * bar * want[n + "_d1"][keep]
        if half and n + "_d" in want:
            own = (2.0 ** -16 if record else 2.0 ** -8) * want[n + "_d"][keep]
            extra = half * want[n + "_d1"][keep] + own + cancelled
        err = (g - w).abs()
        most = half * (w.abs() + size) * (1 + half) + extra + 16 * bar * rms + 1e-30
        print(f"{label}: {n} {float(err.norm()) / max(float(w.norm()), 1e-30):.2e}", flush=True)
        assert (err <= most).all(), f"{label}: {n} off by {float((err / most).max()):.2f} bars"
        two = bar * float(size.norm()) + (float(cancelled.norm()) if n + "_d1" in want else 0.0) + 1e-30
        if half:
            terms = want[n + "_2"][keep] if n + "_2" in want else torch.zeros_like(w)
            two += 1.5 * half * math.sqrt((float(w.norm()) ** 2 + float(terms.norm()) ** 2) / 3)
            if n + "_d" in want:
                two += 1.5 * half / 3 ** 0.5 * float(want[n + "_d2"][keep].norm()) + float(own.norm())
        # with few values a rounding need not be spread evenly
        assert float(err.norm()) <= two or w.numel() < 500, f"{label}: {n} 2-norm off"


def randn(gen, *s):
    return torch.randn(s, generator=gen)


def inputs(B, T, Hq, Hk, D, dtype, *, seed=1, fused=False, size=1.0):
    gen = torch.Generator().manual_seed(seed)
    dy = randn(gen, B, T, Hq, D).to(dtype).cuda()
    if fused:
        x = randn(gen, B, T, Hq + 2 * Hk, D).to(dtype).cuda()
        return dict(q=x[:, :, :Hq], k=x[:, :, Hq:Hq + Hk], v=x[:, :, Hq + Hk:], dy=dy)
    return dict(q=(size * randn(gen, B, T, Hq, D)).to(dtype).cuda(), k=randn(gen, B, T, Hk, D).to(dtype).cuda(),
                v=randn(gen, B, T, Hk, D).to(dtype).cuda(), dy=dy)


def run(d, *, starts=None, scale=None, record=True, **kw):
    st = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    a = [d[n] for n in ("q", "k", "v")]
    y, lse, rec = api.attn_forward(*a, seq_starts=st, scale=scale, want_lse=True, want_record=record, **kw)
    out = api.attn_backward(*a, y, lse, d["dy"], rec, seq_starts=st, scale=scale, **kw)
    return dict(out, y=y, lse=lse)


def reference(d, *, starts=None, scale=None):
    return R.attention(d["q"], d["k"], d["v"], d["dy"], starts=starts, scale=scale)


CASES = [
    # B, T, Hq, Hk, D, dtype, fused, record
    (1, 1, 1, 1, 64, F32, False, True),
    (1, 1, 2, 1, 128, BF16, False, True),
    (2, 2, 3, 1, 64, BF16, False, False),
    (3, 17, 2, 2, 128, F32, True, True),
    (1, 31, 4, 2, 64, BF16, True, True),
    (2, 32, 1, 1, 128, BF16, False, True),
    (1, 33, 8, 1, 64, F32, False, True),
    (1, 63, 2, 1, 64, BF16, False, True),
    (2, 64, 2, 2, 128, BF16, True, False),
    (1, 65, 5, 1, 128, F32, False, True),
    (1, 127, 1, 1, 64, BF16, False, True),
    (2, 128, 4, 2, 128, BF16, False, True),
    (1, 129, 6, 2, 64, F32, True, True),
    (1, 200, 3, 3, 128, BF16, True, True),
    (2, 257, 2, 1, 64, BF16, False, True),
    (1, 500, 2, 1, 128, F32, False, True),
    (1, 777, 4, 1, 128, BF16, False, True),
    (1, 1030, 2, 2, 64, BF16, False, True),
]


@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c)).replace("torch.", "") for c in CASES])
def test_attention(case):
    B, T, Hq, Hk, D, dt, fused, record = case
    print(f"case {case}", flush=True)
    d = inputs(B, T, Hq, Hk, D, dt, fused=fused)
    check(run(d, record=record), reference(d), str(case), D=D, T=T, record=record)


PACKED = [
    ([0, 5], 5, F32, 64), ([0, 0, 1, 1, 40, 104, 104], 104, BF16, 64),
    ([0, 128, 256, 257, 600], 600, BF16, 128), ([3, 130, 131, 390], 400, F32, 128),
    ([10, 10, 10], 20, BF16, 64), ([0] + [3 * i for i in range(1, 80)], 240, BF16, 128),
    ([0, 127, 255, 383, 384], 384, BF16, 64),
]


@pytest.mark.parametrize("case", PACKED, ids=[f"{len(c[0]) - 1}-{c[1]}-{c[2]}-{c[3]}".replace("torch.", "") for c in PACKED])
def test_packed(case):
    """Sequences end to end; rows outside every sequence stay as they were and
    what they hold reaches nothing."""
    starts, T, dt, D = case
    d = inputs(1, T, 4, 2, D, dt, seed=3)
    outside = torch.ones(T, dtype=torch.bool)
    for lo, hi in zip(starts[:-1], starts[1:]):
        outside[lo:hi] = False
    for n in d:
        d[n][:, outside.cuda()] = math.nan
    want = R.attention(*(torch.nan_to_num(d[n]) for n in ("q", "k", "v", "dy")), starts=starts)
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    mark = {n: torch.full_like(d[n], 7.0, memory_format=torch.contiguous_format) for n in ("q", "k", "v")}
    y, lse = torch.full_like(d["q"], 7.0), torch.full(d["q"].shape[:3], 7.0, device="cuda")
    a = [d[n] for n in ("q", "k", "v")]
    _, _, rec = api.attn_forward(*a, seq_starts=st, want_lse=True, want_record=True, out=(y, lse, None))
    g = api.attn_backward(*a, y, lse, d["dy"], rec, seq_starts=st, out={"d" + n: mark[n] for n in mark})
    got = dict(g, y=y, lse=lse)
    for n, x in got.items():
        assert (x[:, outside.cuda()] == 7.0).all(), n
    check(got, want, str(case), D=D, T=max(hi - lo for lo, hi in zip(starts[:-1], starts[1:])) or 1)


def test_many_sequences():
    """More sequences than a wave's lanes, and a slot search that has depth."""
    starts = [0]
    gen = torch.Generator().manual_seed(5)
    for n in torch.randint(0, 9, (700,), generator=gen).tolist():
        starts.append(starts[-1] + n)
    d = inputs(1, starts[-1], 2, 1, 64, BF16, seed=6)
    check(run(d, starts=starts), reference(d, starts=starts), "many", D=64, T=9)


def test_starts_out_of_range():
    """Starts outside [0, T] are clamped to it."""
    d = inputs(1, 100, 2, 1, 64, BF16, seed=7)
    check(run(d, starts=[-50, 40, 2 ** 31 - 1]), reference(d, starts=[0, 40, 100]), "clamped", D=64, T=60)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_scale_and_size(dt):
    """Scores far apart: the running maximum grows by hundreds, and falls."""
    d = inputs(1, 300, 2, 1, 64, dt, seed=8, size=3.0)
    ramp = torch.linspace(-8, 8, 300, device="cuda")[None, :, None, None]
    d["k"] = (d["k"].float() + ramp).to(dt)
    d["q"] = (d["q"].float() + 1).to(dt)
    w = reference(d, scale=0.3)
    # a score's own rounding, relative to its terms' sizes (up to 0.3 * 64 * 8 * 4), is an error of its weight
    got = run(d, scale=0.3)
    check(got, w, "ramp", D=64 * 200, T=300)
    assert torch.isfinite(got["y"]).all()


def test_equal_scores_and_zeros():
    d = inputs(1, 260, 2, 2, 128, BF16, seed=9)
    d["q"].zero_()
    check(run(d), reference(d), "zeros", D=128, T=260)
    lse = run(d)["lse"].cpu().double()
    want = torch.log(torch.arange(1, 261).double())[None, :, None].expand_as(lse)
    assert ((lse - want).abs() <= 2.0 ** -22 * (1 + want)).all()


def test_gradients_against_differences():
    """fp32, along one direction of each input: a central difference of
    sum(dy y) formed from the device's own y in fp64."""
    d = inputs(1, 90, 4, 2, 64, F32, seed=10)
    g = run(d)
    for n in ("q", "k", "v"):
        gen = torch.Generator().manual_seed(11)
        e = randn(gen, *d[n].shape).cuda()

        def value(s):
            y = api.attn_forward(*({**d, n: (d[n].double() + s * e.double()).float()}[m] for m in "qkv"))[0]
            return float((y.double() * d["dy"].double()).sum())

        h = 2.0 ** -7
        diff = (value(h) - value(-h)) / (2 * h)
        want = float((g["d" + n].double() * e.double()).sum())
        # third derivatives: h^2 / 6 of a few times the norms; rounding: 2^-24 sqrt(n) |dy| |y| / h
        tol = h * h * float(e.norm()) * float(d["dy"].norm()) + 2.0 ** -24 * 128 * float(d["dy"].norm()) / h
        assert abs(diff - want) <= tol, (n, diff, want, tol)


def test_nan_in_later_tokens():
    """A key after a token, and 64 tokens and more behind it, reaches nothing,
    whatever it holds; a NaN in k alone never does."""
    d = inputs(1, 400, 2, 1, 64, BF16, seed=12)
    clean = api.attn_forward(d["q"], d["k"], d["v"])[0]
    d["k"][:, 301] = math.nan
    assert torch.equal(api.attn_forward(d["q"], d["k"], d["v"])[0][:, :301], clean[:, :301])
    d["v"][:, 301] = math.inf
    assert torch.equal(api.attn_forward(d["q"], d["k"], d["v"])[0][:, :301 - 63], clean[:, :301 - 63])


WIDE = [
    # B, T, Hq, Hk, D, dtype: enough workgroups of 128 rows for the forms that share the keys
    (8, 130, 16, 16, 64, BF16), (33, 257, 11, 11, 64, BF16), (2, 300, 96, 48, 128, BF16), (3, 389, 24, 8, 128, BF16),
    (16, 200, 32, 16, 64, F32), (6, 257, 32, 32, 128, F32), (1, 1, 520, 520, 64, F32), (257, 1, 2, 1, 128, BF16),
]


@pytest.mark.parametrize("case", WIDE, ids=["-".join(map(str, c)).replace("torch.", "") for c in WIDE])
def test_many_workgroups(case):
    B, T, Hq, Hk, D, dt = case
    print(f"case {case}", flush=True)
    d = inputs(B, T, Hq, Hk, D, dt, fused=B == 3)
    check(run(d), reference(d), str(case), D=D, T=T)


@pytest.mark.parametrize("dt, D, Hq, Hk, nseq", [(BF16, 64, 6, 3, 64), (BF16, 128, 4, 4, 65), (F32, 64, 8, 8, 90),
                                                 (F32, 128, 16, 8, 50), (BF16, 64, 16, 8, 60), (BF16, 128, 8, 8, 64)])
def test_many_workgroups_packed(dt, D, Hq, Hk, nseq):
    gen = torch.Generator().manual_seed(14)
    n = torch.randint(0, 200, (nseq,), generator=gen)
    n[7], n[8], n[20], n[40] = 0, 1, 128, 385
    starts = [5] + (5 + n.cumsum(0)).tolist()
    T = starts[-1] + 9
    d = inputs(1, T, Hq, Hk, D, dt, seed=15)
    check(run(d, starts=starts), reference(d, starts=starts), f"{dt} {D}", D=D, T=385)


@pytest.mark.parametrize("dt, Hq", [(BF16, 1), (F32, 8)])
def test_one_long_sequence_among_short_ones(dt, Hq):
    """More tiles in a sequence than the search for them looks at in one step."""
    starts = [0, 3, 3, 40, 40 + 2090, 2140, 2269]
    d = inputs(1, 2269, Hq, 1, 64, dt, seed=18)
    check(run(d, starts=starts), reference(d, starts=starts), f"{dt}", D=64, T=2090)


def test_nothing_to_do():
    for B, T in ((0, 5), (3, 0), (0, 0)):
        q, k = torch.zeros(B, T, 4, 64, device="cuda"), torch.zeros(B, T, 2, 64, device="cuda")
        y, lse, rec = api.attn_forward(q, k, k, want_lse=True, want_record=True)
        assert y.shape == q.shape and lse.shape == q.shape[:3] and rec is None
        g = api.attn_backward(q, k, k, y, lse, q)
        assert g["dq"].shape == q.shape and g["dk"].shape == k.shape
        w = torch.ones(64, device="cuda")
        assert api.qk_norm_forward(q, k, w, w)[0].shape == q.shape
        g = api.qk_norm_backward(q, k, q, k, w, w)
        assert (g["dwq"] == 0).all() and (g["dwk"] == 0).all()
        c = cache(max(B, 1), 2, 16, 2, 64, F32, F32)
        if B == 0:
            c["table"] = c["table"][:0]
        ln = torch.ones(B, dtype=torch.int32, device="cuda")
        before = c["k_pages"].clone()
        api.kv_write(k, k, *cargs(c, ln))
        assert torch.equal(before, c["k_pages"])
        assert api.kv_read(*cargs(c, ln), T=T)[0].shape == k.shape
        assert api.attn_decode(q, *cargs(c, ln)).shape == q.shape


def test_scores_of_minus_infinity():
    """Keys whose scores are minus infinity have no weight, also where no other
    came before them; a token with no other key has NaN."""
    for dt, B in ((BF16, 1), (F32, 1), (BF16, 130), (F32, 130)):
        d = inputs(B, 200, 2, 1, 64, dt, seed=16)
        d["q"].abs_().add_(0.1)
        d["k"][:, :90] = -math.inf
        y, lse, _ = api.attn_forward(d["q"], d["k"], d["v"], want_lse=True)
        assert torch.isnan(y[:, :90]).all() and (lse[:, :90] == -math.inf).all()
        want = R.attention(d["q"][:, 90:], d["k"][:, 90:], d["v"][:, 90:], d["dy"][:, 90:])
        check(dict(y=y[:, 90:], lse=lse[:, 90:]), want, f"{dt} {B}", D=64, T=200)


def test_offsets_past_32_bits():
    """Parts of rows so wide that the last tokens' elements are past 2^31."""
    x = torch.empty(1, 600, 65536, 64, dtype=BF16, device="cuda")
    d = inputs(1, 600, 4, 2, 64, BF16, seed=17)
    far = dict(q=x[:, :, 40000:40004], k=x[:, :, 65000:65002], v=x[:, :, 65534:], dy=d["dy"])
    for n in "qkv":
        far[n].copy_(d[n])
    a, b = run(d), run(far)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    theta = (10000.0 ** (-torch.arange(0, 64, 2) / 64)).float().cuda()
    w = torch.ones(64, device="cuda")
    for i, j in zip(api.qk_norm_forward(d["q"], d["k"], w, w, theta), api.qk_norm_forward(far["q"], far["k"], w, w, theta)):
        assert torch.equal(i, j)
    g, h = (api.qk_norm_backward(a["dq"], a["dk"], t["q"], t["k"], w, w, theta) for t in (d, far))
    for n in g:
        assert torch.equal(g[n], h[n]), n


def test_same_bits_every_time():
    d = inputs(2, 700, 4, 2, 128, BF16, seed=13)
    a, b = run(d), run(d)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    # a workspace that held something else, other outputs, another stream
    ws = torch.full((api.attn_backward_workspace_bytes(2, 700, 4, 2, 128),), 255, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    args = [d[n] for n in "qkv"]
    y, lse, rec = api.attn_forward(*args, want_lse=True, want_record=True, stream=side)
    c = api.attn_backward(*args, y, lse, d["dy"], rec, workspace=ws, stream=side)
    side.synchronize()
    for n in c:
        assert torch.equal(a[n], c[n]), n


def test_strides_that_are_refused():
    """Tensors that are not tokens at one stride are refused, not misread."""
    x = torch.zeros(2, 6, 4, 64, device="cuda")
    k = torch.zeros(2, 6, 2, 64, device="cuda")
    api.attn_forward(x, k, k)
    wide = torch.zeros(2, 6, 8, 68, device="cuda")
    for bad in (x[:, :1].expand(2, 6, 4, 64), x[:1].expand(2, 6, 4, 64), x[:, :, :1].expand(2, 6, 4, 64),
                torch.zeros(2, 4, 6, 64, device="cuda").transpose(1, 2), torch.zeros(2, 7, 4, 64, device="cuda")[:, :6],
                wide[:, :, :4, :64], torch.zeros(2, 6, 4, 128, device="cuda")[..., ::2], x.half(), x[..., :32], x[0]):
        with pytest.raises(ValueError):
            api.attn_forward(bad, k, k)
    with pytest.raises(ValueError):
        api.attn_forward(x, k, k[:, :5])
    with pytest.raises(ValueError):
        api.attn_forward(x, k, k.cpu())
    with pytest.raises(ValueError):
        api.attn_forward(x[:, :, :3], k, k)
    with pytest.raises(ValueError):
        api.attn_forward(x, k, k, seq_starts=torch.tensor([0, 6], dtype=torch.int32, device="cuda"))
    # one row, or rows end to end, at any other stride of whole tokens is fine
    y = api.attn_forward(torch.zeros(2, 6, 9, 64, device="cuda")[:, :, 1:5], k, torch.zeros(2, 6, 3, 64, device="cuda")[:, :, :2])[0]
    assert (y == 0).all()
    z = torch.randn(1, 12, 4, 64, device="cuda")
    assert torch.equal(api.attn_forward(z[:, ::2], k[:1], k[:1])[0], api.attn_forward(z[:, ::2].contiguous(), k[:1], k[:1])[0])


# ------------------------------------------------------- norm and rotation

def qk_inputs(B, T, Hq, Hk, D, R_, dtype, *, seed=20, far=0):
    gen = torch.Generator().manual_seed(seed)
    x = randn(gen, B, T, Hq + Hk + 1, D).to(dtype).cuda()
    d = dict(q=x[:, :, :Hq], k=x[:, :, Hq:Hq + Hk], wq=(1 + 0.2 * randn(gen, D)).cuda(), wk=(1 + 0.2 * randn(gen, D)).cuda(),
             theta=(10000.0 ** (-torch.arange(0, R_, 2) / max(R_, 1))).float().cuda() if R_ else None,
             positions=(torch.randint(-far, far + 1, (B, T), generator=gen) if far else torch.randint(0, 500, (B, T), generator=gen)).int().cuda(),
             dq=randn(gen, B, T, Hq, D).to(dtype).cuda(), dk=randn(gen, B, T, Hk, D).to(dtype).cuda())
    return d


def qk_run(d, **kw):
    a = [d[n] for n in ("q", "k", "wq", "wk", "theta", "positions")]
    q, k = api.qk_norm_forward(*a, **kw)
    return dict(api.qk_norm_backward(d["dq"], d["dk"], *a, **kw), q=q, k=k)


def qk_check(got, d, label, **kw):
    """fp32: a mean of D squares, a rotation (two products, whose angle is off by
    2^-22 of a turn's part) and the mean of D products: 4 * sqrt(128) * 2^-24
    of the head's size and 2^-20; weights' gradients: sums of n terms, sqrt(n)
    steps of 2^-24 of the root of their squares' sum.  bf16: half a step more."""
    want = R.qk_norm(*(d[n] for n in ("q", "k", "wq", "wk", "theta", "positions", "dq", "dk")), **kw)
    for n in ("q", "k", "dq", "dk"):
        g, w = got[n].cpu().double(), want[n]
        if not w.numel():
            continue
        head = w.norm(dim=-1, keepdim=True)
        most = HALF_STEP[got[n].dtype] * w.abs() + (4 * 128 ** 0.5 * 2.0 ** -24 + 2.0 ** -20) * head + 1e-30
        err = (g - w).abs()
        print(f"{label}: {n} {float(err.norm() / w.norm()):.2e}", flush=True)
        assert (err <= most).all(), f"{label}: {n} {float((err / most).max()):.2f} bars"
    for n in ("dwq", "dwk"):
        if d["wq"] is None:
            assert got[n] is None
            continue
        g, w = got[n].cpu().double(), want[n]
        rows = d["q"].shape[0] * d["q"].shape[1] * d["q"].shape[2]
        most = (rows ** 0.5 + 16) * 2.0 ** -22 * want[n + "_2"] + 1e-30
        assert ((g - w).abs() <= most).all(), f"{label}: {n}"


QK = [
    # B, T, Hq, Hk, D, R, dtype, far
    (1, 1, 1, 1, 64, 64, F32, 0), (2, 3, 5, 1, 128, 128, BF16, 0), (1, 17, 4, 2, 64, 32, BF16, 0),
    (3, 33, 2, 2, 128, 16, F32, 0), (1, 70, 7, 3, 64, 48, F32, 10 ** 6), (2, 1, 16, 4, 128, 64, BF16, 2 ** 31 - 1),
    (1, 1500, 3, 1, 64, 0, BF16, 0), (40, 60, 2, 1, 128, 96, F32, 0), (5, 1, 0, 2, 64, 64, BF16, 0), (2, 2, 3, 0, 64, 64, F32, 0),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", QK, ids=["-".join(map(str, c)).replace("torch.", "") for c in QK])
def test_qk_norm(case, interleaved):
    B, T, Hq, Hk, D, R_, dt, far = case
    d = qk_inputs(B, T, Hq, Hk, D, R_, dt, far=far)
    qk_check(qk_run(d, interleaved=interleaved), d, str(case), interleaved=interleaved)


def test_qk_norm_parts_of_it():
    """Without weights (the rotation alone), without positions, in place."""
    d = qk_inputs(2, 9, 4, 2, 64, 64, F32)
    d["wq"] = d["wk"] = None
    qk_check(qk_run(d), d, "no weights")
    d = qk_inputs(2, 9, 4, 2, 128, 64, BF16)
    d["positions"] = None
    qk_check(qk_run(d, eps=1e-3), d, "no positions", eps=1e-3)
    d = {n: x.contiguous() for n, x in qk_inputs(3, 50, 4, 2, 128, 64, BF16).items()}
    want = qk_run(d)
    a = [d[n] for n in ("wq", "wk", "theta", "positions")]
    q, k = d["q"].clone(), d["k"].clone()
    dq, dk = d["dq"].clone(), d["dk"].clone()
    g = api.qk_norm_backward(dq, dk, q, k, *a, out=dict(dq=dq, dk=dk))
    api.qk_norm_forward(q, k, *a, out=(q, k))
    for n, x in dict(q=q, k=k, dq=dq, dk=dk, dwq=g["dwq"], dwk=g["dwk"]).items():
        assert torch.equal(x, want[n]), n


def test_qk_norm_zero_head():
    """A head of zeros stays zeros; its gradient is that of x / sqrt(eps)."""
    d = qk_inputs(1, 4, 2, 1, 64, 64, F32)
    d["q"][:, 1] = 0
    got = qk_run(d)
    assert (got["q"][:, 1] == 0).all()
    qk_check(got, d, "zeros")


# ------------------------------------------------------------------ the cache

def cache(rows, most, page, Hk, D, dtype, kind, *, seed=30, extra=3):
    gen = torch.Generator().manual_seed(seed)
    pages = rows * most + extra
    table = torch.randperm(pages, generator=gen)[:rows * most].view(rows, most).int().cuda()
    k, v = (randn(gen, pages, Hk, page, D) for _ in range(2))
    if kind is not E4M3:
        return dict(k_pages=k.to(dtype).cuda(), v_pages=v.to(dtype).cuda(), table=table, k_scale=None, v_scale=None)
    out = dict(table=table)
    for n, x in (("k", k), ("v", v)):
        z, s = R.quantise(x)
        out[n + "_pages"], out[n + "_scale"] = z.float().to(E4M3).cuda(), s.cuda()
    return out


def dense(c, n):
    """A cache's values in fp64, on the CPU."""
    x = c[n + "_pages"].cpu().float().double()
    return x if c[n + "_scale"] is None else x * c[n + "_scale"].cpu().double()[..., None]


def cargs(c, lens):
    return [c["k_pages"], c["v_pages"], c["table"], lens, c["k_scale"], c["v_scale"]]


CACHES = [
    # rows, T or starts, most, page, Hk, D, dtype, kind, lens
    (2, 1, 3, 16, 1, 64, F32, F32, [48, 1]),
    (3, 4, 2, 32, 2, 128, BF16, BF16, [64, 2, 0]),
    (2, 20, 4, 16, 3, 64, BF16, E4M3, [64, 33]),
    (4, [0, 0, 40, 41, 100], 2, 64, 2, 128, BF16, E4M3, [7, 128, 1, 90]),
    (2, [2, 30, 33], 1, 256, 1, 128, F32, E4M3, [28, 200]),
    (3, [0, 10, 10, 25], 3, 16, 5, 64, F32, F32, [100, 5, -3]),
]


@pytest.mark.parametrize("case", CACHES, ids=["-".join(map(str, c[2:8])).replace("torch.", "") for c in CACHES])
def test_cache(case):
    """Writes are the oracle's values bit for bit, nothing else changes, and
    reads return them (rounded once)."""
    rows, T, most, page, Hk, D, dt, kind, lens = case
    c = cache(rows, most, page, Hk, D, dt, kind)
    if rows == 4:
        c["table"][3, 0] = 10 ** 6          # a page that is not there
        c["table"][1, 1] = -1
    starts = T if isinstance(T, list) else None
    counts = [b - a for a, b in zip(starts[:-1], starts[1:])] if starts else [T] * rows
    B, n = (1, starts[-1] + 2) if starts else (rows, T)
    gen = torch.Generator().manual_seed(31)
    x = randn(gen, B, n, 2 * Hk + 1, D).to(dt).cuda()
    x[0, -1 if not starts else starts[0], 0] = 0      # a head of zeros
    x[0, 0 if not starts else starts[0] + 1, 0, 5] = 1e-30
    k, v = x[:, :, :Hk], x[:, :, Hk:2 * Hk]
    st = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    pages = c["k_pages"].shape[0]
    want = {m: dense(c, m) for m in "kv"}
    where = R.places(lens, counts, c["table"].tolist(), page, pages)
    read = {m: torch.full((B, n, Hk, D), math.nan, dtype=torch.float64) for m in "kv"}
    for r, row in enumerate(where):
        for i, at in enumerate(row):
            b, t = (0, starts[r] + i) if starts else (r, i)
            for m, src in (("k", k), ("v", v)):
                val = src[b, t].cpu()
                if kind is E4M3:
                    z, s = R.quantise(val)
                    val = z * s.double()[:, None]
                val = val.double()
                if at is None:
                    read[m][b, t] = 0
                    continue
                want[m][at[0], :, at[1]] = val
                read[m][b, t] = val
    api.kv_write(k, v, *cargs(c, ln), seq_starts=st)
    for m in "kv":
        assert torch.equal(dense(c, m), want[m]), m
    out = tuple(torch.full((B, n, Hk, D), 7.0, dtype=dt, device="cuda") for _ in range(2))
    got = api.kv_read(*cargs(c, ln), T=n, seq_starts=st, dtype=dt, out=out)
    for m, g in zip("kv", got):
        w = read[m].float().to(dt).double()
        w = torch.where(torch.isnan(read[m]), 7.0, w)
        assert torch.equal(g.cpu().double(), w), m


def test_cache_in_8_bits():
    """Every e4m3 value, ties and values between, and heads that hold what is
    not finite."""
    codes = torch.arange(256, dtype=torch.uint8).view(E4M3).float()
    vals = codes[torch.isfinite(codes)].double().unique()
    mids = (vals[1:] + vals[:-1]) / 2
    x = torch.cat((vals, mids, torch.nextafter(mids.float(), torch.tensor(1e9)).double(),
                   torch.nextafter(mids.float(), torch.tensor(-1e9)).double()))
    n = -(-x.numel() // 63)
    heads = torch.zeros(n, 64)
    heads[:, 0] = 448.0                       # the scale is 1
    flat = torch.zeros(n * 63)
    flat[:x.numel()] = x.float()
    heads[:, 1:] = flat.view(n, 63)
    heads = torch.cat((heads, heads[:3]))
    heads[-3, 7], heads[-2, 9], heads[-1, 1] = math.nan, math.inf, -math.inf
    n = heads.shape[0]
    k = heads.view(1, n, 1, 64).cuda()
    c = dict(k_pages=torch.zeros(2, 1, 256, 64, device="cuda").to(E4M3), table=torch.tensor([[1, 0]], dtype=torch.int32, device="cuda"))
    c.update(v_pages=c["k_pages"].clone(), k_scale=torch.zeros(2, 1, 256, device="cuda"), v_scale=torch.zeros(2, 1, 256, device="cuda"))
    ln = torch.tensor([n], dtype=torch.int32, device="cuda")
    api.kv_write(k, k, *cargs(c, ln))
    got, _ = api.kv_read(*cargs(c, ln), T=n, dtype=F32)
    got = got.cpu().double().view(n, 64)
    assert torch.equal(got[:-3], R.e4m3(heads[:-3].double()))
    assert torch.isnan(got[-3:]).all()


# -------------------------------------------------------------- decode

DECODE = [
    # B, T, Hq, Hk, D, page, most, dtype, kind, lens
    (1, 1, 1, 1, 64, 16, 1, F32, F32, [1]),
    (2, 1, 4, 2, 128, 16, 5, BF16, BF16, [80, 33]),
    (3, 1, 8, 1, 64, 32, 3, BF16, E4M3, [96, 0, 7]),
    (2, 3, 6, 2, 128, 64, 4, F32, F32, [200, 2]),
    (2, 5, 12, 1, 64, 16, 9, BF16, BF16, [144, 131]),     # 60 rows of queries: two tiles
    (1, 2, 40, 1, 128, 256, 2, BF16, E4M3, [512]),
    (4, 1, 3, 3, 64, 128, 30, F32, E4M3, [3840, 1, 2000, -5]),
    (2, 1, 2, 1, 128, 16, 300, BF16, BF16, [4800, 4790]),  # many parts
    (1, 1, 16, 2, 64, 64, 64, BF16, E4M3, [4000]),
]


def decode_bar(want, D, T, dt, kind):
    """As above; a weight is rounded to 2^-16 of itself (two bf16 parts), over an
    8-bit cache to 2^-8 (one)."""
    weight = 0.0 if dt is F32 else 2.0 ** -8 if kind is E4M3 else 2.0 ** -16
    bar = 2 * 6 * max(D, T) ** 0.5 * 2.0 ** -24
    return (HALF_STEP[dt] * (want["y"].abs() + weight * want["y_1"]) + weight * want["y_1"]
            + 16 * bar * (want["y_1"] ** 2).mean().sqrt() + 1e-30)


@pytest.mark.parametrize("case", DECODE, ids=["-".join(map(str, c[:9])).replace("torch.", "") for c in DECODE])
def test_decode(case):
    B, T, Hq, Hk, D, page, most, dt, kind, lens = case
    c = cache(B, most, page, Hk, D, dt, kind)
    # what lies behind a row's end in its pages, and in nobody's pages, may be anything
    for b, n in enumerate(lens):
        for pos in range(max(n, 0), most * page):
            p, o = int(c["table"][b, pos // page]), pos % page
            for m in "kv":
                if kind is E4M3:
                    c[m + "_pages"].view(torch.uint8)[p, :, o] = 0x7F
                    c[m + "_scale"][p, :, o] = math.nan
                else:
                    c[m + "_pages"][p, :, o] = math.nan
            if pos > n + 300:
                break
    gen = torch.Generator().manual_seed(32)
    q = randn(gen, B, T, Hq + 2, D).to(dt).cuda()[:, :, 1:-1]
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    y = api.attn_decode(q, *cargs(c, ln))
    want = R.decode(q, dense(c, "k"), dense(c, "v"), c["table"].tolist(), lens)
    err = (y.cpu().double() - want["y"]).abs()
    most_ = decode_bar(want, D, max(lens), dt, kind)
    print(f"{case}: {float(err.norm() / want['y'].norm()):.2e}", flush=True)
    assert (err <= most_).all(), float((err / most_).max())
    for b, n in enumerate(lens):
        if n <= 0:
            assert (y[b] == 0).all()
    assert torch.equal(y, api.attn_decode(q, *cargs(c, ln)))


@pytest.mark.parametrize("kind", [BF16, E4M3])
def test_decode_bad_pages(kind):
    """Pages that are not in the pool are seen by nobody, lengths past the
    table end with it."""
    c = cache(3, 4, 16, 2, 64, BF16, kind, seed=33)
    c["table"][0, 1] = -1
    c["table"][0, 2] = 2 ** 31 - 1
    c["table"][1] = c["k_pages"].shape[0]
    lens = [64, 40, 1000]
    gen = torch.Generator().manual_seed(34)
    q = randn(gen, 3, 2, 4, 64).to(BF16).cuda()
    y = api.attn_decode(q, *cargs(c, torch.tensor(lens, dtype=torch.int32, device="cuda")))
    want = R.decode(q, dense(c, "k"), dense(c, "v"), c["table"].tolist(), lens)
    assert (y[1] == 0).all()
    assert ((y.cpu().double() - want["y"]).abs() <= decode_bar(want, 64, 64, BF16, kind)).all()


@pytest.mark.parametrize("kind", [F32, E4M3])
def test_decode_many_tokens(kind):
    """More new tokens than a workgroup has; what a later one holds does not reach
    those 64 before it, and a token's NaN stays its own."""
    T, n = 150, 331
    c = cache(2, 24, 16, 2, 64, F32, kind, seed=37)
    gen = torch.Generator().manual_seed(38)
    q = randn(gen, 2, T, 6, 64).cuda()
    lens = [n, 100]         # the second row's first 50 tokens see nothing
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    y = api.attn_decode(q, *cargs(c, ln))
    want = R.decode(q, dense(c, "k"), dense(c, "v"), c["table"].tolist(), lens)
    assert ((y.cpu().double() - want["y"]).abs() <= decode_bar(want, 64, n, F32, kind)).all()
    assert (y[1, :50] == 0).all()
    page, at = int(c["table"][0, 320 // 16]), 320 % 16
    if kind is E4M3:
        c["v_scale"][page, :, at] = math.nan
    else:
        c["v_pages"][page, :, at] = math.nan
    q[0, 3, 1] = math.nan
    z = api.attn_decode(q, *cargs(c, ln))
    assert torch.isnan(z[0, T - (n - 320):]).all() and torch.isnan(z[0, 3, 1]).all()
    z[0, 3, 1] = y[0, 3, 1]
    keep = T - (n - 320) - 64
    assert torch.equal(z[0, :keep], y[0, :keep]) and torch.equal(z[1], y[1])


@pytest.mark.parametrize("dt", [BF16, F32])
def test_decode_scores_of_minus_infinity(dt):
    c = cache(1, 9, 32, 1, 64, dt, dt, seed=39)
    k = torch.zeros(1, 288, 1, 64, dtype=dt, device="cuda")
    gen = torch.Generator().manual_seed(40)
    k.copy_(randn(gen, 1, 288, 1, 64))
    v = randn(gen, 1, 288, 1, 64).to(dt).cuda()
    q = (randn(gen, 1, 1, 4, 64).abs() + 0.1).to(dt).cuda()
    ln = torch.tensor([288], dtype=torch.int32, device="cuda")
    api.kv_write(k, v, *cargs(c, ln))
    for b in c["table"][0, :5].tolist():
        c["k_pages"][b] = -math.inf
    y = api.attn_decode(q, *cargs(c, ln))
    want = R.decode(q, dense(c, "k"), dense(c, "v"), [[-1] * 5 + c["table"][0, 5:].tolist()], [288])
    assert ((y.cpu().double() - want["y"]).abs() <= decode_bar(want, 64, 288, dt, dt)).all()


@pytest.mark.parametrize("kind", [BF16, E4M3])
def test_cache_past_32_bits(kind):
    """Pages whose elements lie past 2^31 in the pool."""
    Hk, D, page, pages = 8, 128, 256, 2 ** 13 + 40
    shape = (pages, Hk, page, D)
    c = dict(k_pages=torch.empty(shape, dtype=kind, device="cuda"), v_pages=torch.empty(shape, dtype=kind, device="cuda"),
             k_scale=None, v_scale=None)
    if kind is E4M3:
        c.update({m: torch.empty(shape[:3], device="cuda") for m in ("k_scale", "v_scale")})
    c["table"] = torch.arange(pages - 6, pages, dtype=torch.int32, device="cuda").view(2, 3)
    gen = torch.Generator().manual_seed(42)
    k, v = (randn(gen, 2, 600, Hk, D).to(BF16).cuda() for _ in range(2))
    q = randn(gen, 2, 1, 16, D).to(BF16).cuda()
    ln = torch.tensor([600, 600], dtype=torch.int32, device="cuda")
    small = {m: x if x is None else x[-6:].clone() for m, x in c.items()}
    small["table"] = c["table"] - (pages - 6)
    out = []
    for x in (c, small):
        api.kv_write(k, v, *cargs(x, ln))
        out.append((*api.kv_read(*cargs(x, ln), T=600, dtype=BF16), api.attn_decode(q, *cargs(x, ln))))
    for a, b in zip(*out):
        assert torch.equal(a, b)
    if kind is BF16:
        assert torch.equal(out[0][0], k) and torch.equal(out[0][1], v)


def test_decode_shared_pages():
    """Two rows with one prefix: the same pages in both rows of the table."""
    c = cache(2, 4, 16, 1, 64, BF16, BF16, seed=35)
    c["table"][1, :2] = c["table"][0, :2]
    gen = torch.Generator().manual_seed(36)
    q = randn(gen, 1, 1, 2, 64).to(BF16).cuda().expand(2, 1, 2, 64).contiguous()
    y = api.attn_decode(q, *cargs(c, torch.tensor([32, 32], dtype=torch.int32, device="cuda")))
    assert torch.equal(y[0], y[1])


# ---------------------------------------------------- a run of them together

@pytest.mark.parametrize("kind", [BF16, E4M3])
def test_prompt_then_tokens(kind):
    """Prompts packed end to end, then three tokens of each: norm and rotation,
    into the cache, attention.  What the last tokens get over the cache is what
    the whole sequences get at once, up to what 8 bits hold."""
    Hq, Hk, D, page = 4, 2, 64, 16
    prompts, more = [37, 1, 64], 3
    total = [n + more for n in prompts]
    gen = torch.Generator().manual_seed(40)
    seqs = [randn(gen, n, Hq + 2 * Hk, D).to(BF16) for n in total]
    theta = (10000.0 ** (-torch.arange(0, D, 2) / D)).float().cuda()
    w = (1 + 0.1 * randn(gen, D)).cuda()

    def layer(x, positions):
        x = x.cuda()
        q, k = api.qk_norm_forward(x[:, :, :Hq], x[:, :, Hq:Hq + Hk], w, w, theta, positions.int().cuda())
        return q, k, x[:, :, Hq + Hk:]

    def starts(ns):
        return torch.tensor([0] + torch.tensor(ns).cumsum(0).tolist(), dtype=torch.int32, device="cuda")

    whole = layer(torch.cat(seqs)[None], torch.cat([torch.arange(n) for n in total])[None])
    want = api.attn_forward(*whole, seq_starts=starts(total))[0]
    c = cache(3, 5, page, Hk, D, BF16, kind, seed=41)
    q, k, v = layer(torch.cat([s[:n] for s, n in zip(seqs, prompts)])[None],
                    torch.cat([torch.arange(n) for n in prompts])[None])
    lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    api.kv_write(k, v, *cargs(c, lens), seq_starts=starts(prompts))
    y = api.attn_forward(q, k, v, seq_starts=starts(prompts))[0]
    for i, n in enumerate(prompts):
        a, b = sum(prompts[:i]), sum(total[:i])
        assert torch.equal(y[:, a:a + n], want[:, b:b + n])
    if kind is BF16:
        back = api.kv_read(*cargs(c, lens), T=sum(prompts), seq_starts=starts(prompts))
        assert torch.equal(back[0], k) and torch.equal(back[1], v)
    for t in range(more):
        x = torch.stack([s[n + t] for s, n in zip(seqs, prompts)])[:, None]
        q, k, v = layer(x, torch.tensor(prompts)[:, None] + t)
        lens = lens + 1
        api.kv_write(k, v, *cargs(c, lens))
        y = api.attn_decode(q, *cargs(c, lens))
        for i, n in enumerate(prompts):
            if kind is BF16:   # two roundings of y and one of the weights, each half a step of at most |v| <= 5
                ref = want[0, sum(total[:i]) + n + t].double()
                assert float((y[i, 0].double() - ref).abs().max()) <= 3 * 2.0 ** -8 * 5
        ref = R.decode(q, dense(c, "k"), dense(c, "v"), c["table"].tolist(), lens.tolist())
        assert ((y.cpu().double() - ref["y"]).abs() <= decode_bar(ref, D, 67, BF16, kind)).all()


def test_captured_and_replayed():
    """A decode step in a graph, replayed with other tokens, lengths and pages."""
    Hq, Hk, D, page = 8, 2, 128, 16
    c = cache(4, 40, page, Hk, D, BF16, BF16, seed=50)
    gen = torch.Generator().manual_seed(51)
    theta = (10000.0 ** (-torch.arange(0, D, 2) / D)).float().cuda()
    w = torch.ones(D, device="cuda")
    x = randn(gen, 4, 1, Hq + 2 * Hk, D).to(BF16).cuda()
    lens = torch.tensor([600, 17, 1, 333], dtype=torch.int32, device="cuda")
    y = torch.empty(4, 1, Hq, D, dtype=BF16, device="cuda")
    ws = torch.empty(api.attn_decode_workspace_bytes(4, 1, Hq, Hk, D, c["k_pages"].shape[0], page, 40),
                     dtype=torch.uint8, device="cuda")

    def step(out):
        q, k = api.qk_norm_forward(x[:, :, :Hq], x[:, :, Hq:Hq + Hk], w, w, theta, lens[:, None])
        api.kv_write(k, x[:, :, Hq + Hk:], *cargs(c, lens))
        return api.attn_decode(q, *cargs(c, lens), workspace=ws, out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(y)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(y)
    for i in range(4):
        x.copy_(randn(gen, 4, 1, Hq + 2 * Hk, D))
        lens += 1 + i
        pages = {n: c[n].clone() for n in ("k_pages", "v_pages")}
        graph.replay()
        got = y.clone()
        after = {n: c[n].clone() for n in pages}
        for n in pages:
            c[n].copy_(pages[n])
        want = step(torch.empty_like(y))
        torch.cuda.synchronize()
        assert torch.equal(got, want), i
        for n in pages:
            assert torch.equal(after[n], c[n]), (i, n)


def test_training_step_captured():
    """Norm, attention and both backwards in a graph, against the eager calls."""
    d = inputs(2, 300, 4, 2, 64, BF16, seed=52, fused=True)
    w = torch.ones(64, device="cuda")
    theta = (10000.0 ** (-torch.arange(0, 64, 2) / 64)).float().cuda()

    def step():
        a = (d["q"], d["k"], w, w, theta)
        q, k = api.qk_norm_forward(*a)
        y, lse, rec = api.attn_forward(q, k, d["v"], want_lse=True, want_record=True)
        g = api.attn_backward(q, k, d["v"], y, lse, d["dy"], rec)
        return dict(api.qk_norm_backward(g["dq"], g["dk"], *a), dv=g["dv"], y=y)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(3):
        gen = torch.Generator().manual_seed(60 + i)
        d["dy"].copy_(randn(gen, *d["dy"].shape))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(got[n], want[n]), (i, n)


def test_graphs_that_share_a_workspace():
    """Two captured calls with one workspace, replayed in turn with eager calls between."""
    c = cache(4, 40, 16, 2, 64, BF16, BF16, seed=70)
    gen = torch.Generator().manual_seed(71)
    q = [randn(gen, 4, 1 + i, 8, 64).to(BF16).cuda() for i in range(2)]
    d = inputs(2, 200, 4, 2, 64, BF16, seed=72)
    lens = torch.tensor([600, 17, 3, 333], dtype=torch.int32, device="cuda")
    need = max(*(api.attn_decode_workspace_bytes(4, 1 + i, 8, 2, 64, c["k_pages"].shape[0], 16, 40) for i in range(2)),
               api.attn_backward_workspace_bytes(2, 200, 4, 2, 64))
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    args = [d[n] for n in "qkv"]
    y, lse, rec = api.attn_forward(*args, want_lse=True, want_record=True)
    calls = [lambda: dict(y=api.attn_decode(q[0], *cargs(c, lens), workspace=ws)),
             lambda: dict(y=api.attn_decode(q[1], *cargs(c, lens), workspace=ws)),
             lambda: api.attn_backward(*args, y, lse, d["dy"], rec, workspace=ws)]
    want = [{n: x.clone() for n, x in f().items()} for f in calls]
    graphs, got = [], []
    for f in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(f())
        graphs.append(g)
    for i in range(6):
        ws.fill_(255)
        for j in ((i, i + 1, i + 2, i) if i % 2 else (i + 2, i)):
            graphs[j % 3].replay()
            for n in want[j % 3]:
                assert torch.equal(got[j % 3][n], want[j % 3][n]), (i, j, n)
                got[j % 3][n].zero_()
        assert torch.equal(calls[i % 2]()["y"], want[i % 2]["y"])


def test_two_streams_at_once():
    d = [inputs(2, 900, 8, 4, 64, BF16, seed=80 + i) for i in range(2)]
    want = [run(x) for x in d]
    c = cache(3, 60, 16, 2, 128, BF16, BF16, seed=82)
    gen = torch.Generator().manual_seed(83)
    q = randn(gen, 3, 1, 8, 128).to(BF16).cuda()
    lens = torch.tensor([900, 17, 400], dtype=torch.int32, device="cuda")
    y = api.attn_decode(q, *cargs(c, lens))
    streams = [torch.cuda.Stream() for _ in d]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for x, s in zip(d, streams):
            with torch.cuda.stream(s):
                got.append((run(x), api.attn_decode(q, *cargs(c, lens))))
    torch.cuda.synchronize()
    for i, (g, z) in enumerate(got):
        assert torch.equal(z, y), i
        for n in g:
            assert torch.equal(g[n], want[i % 2][n]), (i, n)
