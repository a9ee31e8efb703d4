"""The gated delta rule, its epilogue and the residual norm on the device
against the fp64 oracle (oracle.gdr), MI355X only.

Bar.  A value of the recurrence passes through about six sums of at most 128
products (the answers of the state, the triangular solve, the read-out, the
update; the gradients as many again).  Rounding errors of such a sum add up
like a random walk, sqrt(128) steps of 2^-24 of the sum's size, so the
2-norm of the error may reach 2 * 6 * sqrt(128) * 2^-24 < 8.1e-6 of the result's,
and a single element 16 times the RMS of that (its own share of the largest
terms).  Outputs in bf16 are rounded once: half a step, 2^-8 of the element
at most, 2^-8 in the 2-norm."""
import pytest
import torch

import oracle.gdr as R
from linear_attention_rnn_wkv7_amd import api

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
REL = 2 * 6 * 128 ** 0.5 * 2.0 ** -24
HALF_STEP = {F32: 0.0, BF16: 2.0 ** -8}


def check(got, want, label, terms=None):
    """terms: 2-norms of the terms that an output is the difference of, where
    they may cancel: the rounding errors are relative to those."""
    for n, w in want.items():
        if got.get(n) is None:
            continue
        g = got[n].detach().cpu().double()
        assert g.shape == w.shape, (label, n, g.shape, w.shape)
        keep = ~torch.isnan(w)
        g, w = g[keep], w[keep]
        if w.numel() == 0:
            continue
        half = HALF_STEP[got[n].dtype]
        err = (g - w).abs()
        assert torch.isfinite(g).all(), f"{label}: {n} is not finite"
        size = max(float(w.norm()), (terms or {}).get(n, 0.0), 1e-30)
        rms = size / w.numel() ** 0.5
        rel = float((g - w).norm()) / size
        print(f"{label}: {n} {rel:.2e}", flush=True)
        assert rel <= REL + half or float(w.norm()) < 1e-25, f"{label}: {n} off by {rel:.2e}"
        assert (err <= half * w.abs() + 16 * REL * rms + 1e-30).all(), f"{label}: {n} element"


def inputs(B, T, Hk, Hv, K, V, dtype, *, norm=False, s0=True, dsT=True, starts=None, seed=1, decay=0.2):
    gen = torch.Generator().manual_seed(seed)

    def rn(*s):
        return torch.randn(s, generator=gen)

    k = rn(B, T, Hk, K)
    if not norm:
        k = k / k.norm(dim=-1, keepdim=True)
    seqs = B if starts is None else len(starts) - 1
    d = dict(q=rn(B, T, Hk, K).to(dtype), k=k.to(dtype), v=rn(B, T, Hv, V).to(dtype),
             g=-decay * torch.nn.functional.softplus(3 * rn(B, T, Hv)), beta=torch.sigmoid(2 * rn(B, T, Hv)),
             s0=0.3 * rn(seqs, Hv, V, K) if s0 else None, dy=rn(B, T, Hv, V).to(dtype),
             dsT=rn(seqs, Hv, V, K) if dsT else None)
    return {n: None if x is None else x.cuda() for n, x in d.items()}


IN = ("q", "k", "v", "g", "beta")


def run(d, *, starts=None, norm=False, record=True, scale=None, **kw):
    st = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    a = [d[n] for n in IN]
    y, sT, ck = api.gdr_forward(*a, d["s0"], seq_starts=st, norm_qk=norm, want_ckpt=record, scale=scale, **kw)
    out = api.gdr_backward(*a, d["dy"], d["s0"], d["dsT"], ck, seq_starts=st, norm_qk=norm, scale=scale, **kw)
    return dict(out, y=y, sT=sT)


def reference(d, *, starts=None, norm=False, scale=None):
    return R.rule(*(d[n] for n in IN), d["s0"], d["dy"], d["dsT"], starts=starts, norm_qk=norm, scale=scale)


CASES = [
    # B, T, Hk, Hv, K, V, dtype, norm, s0, dsT, record
    (1, 1, 1, 1, 64, 16, F32, False, True, True, True),
    (2, 1, 1, 2, 128, 64, BF16, True, True, True, False),
    (1, 2, 1, 3, 64, 64, F32, False, False, True, True),
    (1, 15, 2, 2, 64, 48, BF16, True, False, False, True),
    (1, 16, 1, 1, 128, 128, F32, True, True, True, False),
    (2, 17, 1, 2, 64, 128, BF16, False, True, False, True),
    (1, 33, 1, 1, 64, 32, F32, False, True, True, True),
    (1, 63, 2, 4, 128, 16, BF16, False, True, True, True),
    (1, 64, 1, 1, 64, 64, BF16, True, True, True, False),
    (2, 65, 2, 2, 64, 64, F32, True, False, False, True),
    (1, 127, 1, 2, 128, 112, F32, True, True, True, True),
    (1, 128, 1, 1, 64, 256, BF16, False, True, True, True),
    (1, 130, 1, 3, 128, 128, BF16, True, True, True, True),
    (3, 200, 2, 2, 64, 80, F32, False, True, True, False),
    (1, 400, 1, 1, 128, 144, BF16, False, False, True, True),
    (1, 777, 2, 2, 64, 64, BF16, True, True, True, True),
]


@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c)).replace("torch.", "") for c in CASES])
def test_rule(case):
    B, T, Hk, Hv, K, V, dt, norm, s0, dsT, record = case
    print(f"case {case}", flush=True)
    d = inputs(B, T, Hk, Hv, K, V, dt, norm=norm, s0=s0, dsT=dsT)
    check(run(d, norm=norm, record=record), reference(d, norm=norm), str(case))


SEGMENTS = [   # rows of 16 chunks and more with few heads run in segments
    (1, 1024, 1, 1, 64, 16, F32, True, True, True, True),
    (1, 1030, 1, 2, 64, 48, BF16, False, True, True, False),
    (2, 1500, 1, 3, 128, 64, BF16, True, True, True, True),
    (1, 1217, 2, 2, 128, 32, F32, False, False, False, True),
    (1, 2100, 1, 1, 64, 64, BF16, True, False, True, True),
]


@pytest.mark.parametrize("case", SEGMENTS, ids=["-".join(map(str, c)).replace("torch.", "") for c in SEGMENTS])
def test_rule_segments(case):
    test_rule(case)


PACKED = [
    [0, 5],
    [0, 0, 1, 65, 65, 130, 131],
    [3, 64, 128, 128, 192, 193],         # rows before the first and behind the last
    [0, 63, 127, 192, 256, 321],         # chunk edges in every place
    [7, 7, 7],                           # nothing but empty ones
    list(range(0, 41)),                  # one token each
]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("starts", PACKED, ids=[str(i) for i in range(len(PACKED))])
def test_rule_packed(starts, dt):
    T = starts[-1] + 9
    print(f"packed {starts} {dt}", flush=True)
    d = inputs(1, T, 1, 2, 64, 48, dt, starts=starts, norm=True)
    for n in IN + ("dy",):   # tokens outside the sequences are not read ..
        d[n][:, :starts[0]] = float("nan")
        d[n][:, starts[-1]:] = float("nan")
    mark = {n: torch.full_like(d[n], 7.0) for n in IN}
    y = torch.full_like(d["v"], 7.0)
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    a = [d[n] for n in IN]
    _, sT, ck = api.gdr_forward(*a, d["s0"], seq_starts=st, norm_qk=True, want_ckpt=True, out=(y, None, None))
    out = api.gdr_backward(*a, d["dy"], d["s0"], d["dsT"], ck, seq_starts=st, norm_qk=True,
                           out={"d" + n: mark[n] for n in IN})
    got = dict(out, y=y, sT=sT)
    check(got, reference(d, starts=starts, norm=True), str(starts))
    for n in ("y",) + tuple("d" + n for n in IN):   # .. nor written
        assert (got[n][:, :starts[0]] == 7).all() and (got[n][:, starts[-1]:] == 7).all(), n


def test_rule_starts_out_of_range():
    """Starts outside [0, T] are clamped to it."""
    d = inputs(1, 100, 1, 1, 64, 16, F32, starts=[0, 40, 100])
    a = [d[n] for n in IN]
    ok, bad = (torch.tensor(s, dtype=torch.int32, device="cuda") for s in ([0, 40, 100], [-5, 40, 2 ** 31 - 1]))
    y0, s0, _ = api.gdr_forward(*a, d["s0"], seq_starts=ok)
    y1, s1, _ = api.gdr_forward(*a, d["s0"], seq_starts=bad)
    assert torch.equal(y0, y1) and torch.equal(s0, s1)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_rule_extreme_gates(dt):
    """Decays of 0 (log -inf, -1e30, -200) and of 1, beta of 0 and 1, keys that
    are all alike, keys and queries of zeros under the norm."""
    d = inputs(1, 150, 1, 2, 64, 32, dt, norm=True)
    g, be = d["g"], d["beta"]
    g[:, 10:30:4] = -float("inf")
    g[:, 70, 0] = -1e30
    g[:, 71, 0] = -200.0
    g[:, 90:128, 1] = 0.0
    be[:, 20:40] = 0.0
    be[:, 90:110] = 1.0
    d["k"][:, 80:128] = d["k"][:, 80:81]
    d["k"][:, 5] = 0
    d["q"][:, 6] = 0
    check(run(d, norm=True), reference(d, norm=True), f"gates {dt}")


def test_rule_slow_decay_alike_keys():
    """No decay, unit keys all alike, beta 1: (I + L)^-1 of ones, whose powers
    would be binomials."""
    d = inputs(1, 128, 1, 1, 64, 16, F32)
    d["g"].zero_()
    d["beta"].fill_(1.0)
    d["k"][:] = d["k"][:, :1]
    check(run(d), reference(d), "alike")


def test_rule_nothing_leaks_between_sequences():
    """inf and NaN in one sequence stay there."""
    starts = [0, 30, 100, 170]
    d = inputs(1, 170, 1, 1, 64, 16, F32, starts=starts)
    clean = run(d, starts=starts)
    for n, x in (("v", float("inf")), ("q", float("nan")), ("dy", float("inf")), ("g", float("nan"))):
        d[n][:, 40] = x
    got = run(d, starts=starts)
    for n in ("y",) + tuple("d" + m for m in IN):
        for lo, hi in ((0, 30), (100, 170)):
            assert torch.equal(got[n][:, lo:hi], clean[n][:, lo:hi]), n
    for n in ("sT", "ds0"):
        assert torch.equal(got[n][0], clean[n][0]) and torch.equal(got[n][2], clean[n][2])
    assert torch.isnan(got["y"][0, 40]).all() and not torch.isfinite(got["sT"][1]).any()


@pytest.mark.parametrize("dt,K,V", [(F32, 64, 64), (BF16, 128, 48)])
def test_rule_same_bits_again(dt, K, V):
    d = inputs(2, 300, 2, 4, K, V, dt, norm=True)
    a, b = run(d, norm=True), run(d, norm=True, record=False)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    # the parts alone
    args = [d[n] for n in IN]
    y, _, ck = api.gdr_forward(*args, d["s0"], norm_qk=True, want_sT=False)
    assert torch.equal(y, a["y"]) and ck is None
    _, sT, _ = api.gdr_forward(*args, d["s0"], norm_qk=True, want_y=False)
    assert torch.equal(sT, a["sT"])


def test_rule_scale_and_no_tokens():
    d = inputs(1, 70, 1, 1, 64, 16, F32)
    check(run(d, scale=-1.7), reference(d, scale=-1.7), "scale")
    d = inputs(2, 0, 1, 2, 64, 32, BF16)
    got = run(d)
    assert got["y"].shape == (2, 0, 2, 32)
    assert torch.equal(got["sT"], d["s0"]) and torch.equal(got["ds0"], d["dsT"])
    d = inputs(2, 0, 1, 2, 64, 32, BF16, s0=False, dsT=False)
    got = run(d)
    assert not got["sT"].any() and not got["ds0"].any()


def test_rule_other_stream_and_workspace():
    d = inputs(1, 140, 1, 2, 64, 32, BF16)
    want = run(d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run(d, stream=s)
    s.synchronize()
    for n in want:
        assert torch.equal(got[n], want[n]), n
    a = [d[n] for n in IN]
    need = api.gdr_backward_workspace_bytes(1, 140, 1, 2, 64, 32, BF16, ckpt_provided=False)
    ws = torch.empty(need, device="cuda", dtype=torch.uint8)
    got = api.gdr_backward(*a, d["dy"], d["s0"], d["dsT"], workspace=ws)
    for n in got:
        assert torch.equal(got[n], want[n]), n
    with pytest.raises(Exception, match="workspace"):
        api.gdr_backward(*a, d["dy"], d["s0"], d["dsT"], workspace=ws[:need - 256])


def test_rule_captured_twice():
    """Two captured graphs of forward and backward (their own workspaces),
    replayed in turn with eager work between."""
    d = [inputs(1, 100 + 60 * i, 1, 2, 64, 32, (F32, BF16)[i], seed=5 + i) for i in range(2)]
    want = [run(x) for x in d]
    side, graphs, got = torch.cuda.Stream(), [], []
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for x in d:
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=side):
                got.append(run(x))
            graphs.append(gr)
    torch.cuda.synchronize()
    for turn in range(4):
        for i in (0, 1) if turn % 2 else (1, 0):
            for x in got[i].values():
                x.zero_()
            graphs[i].replay()
            eager = run(d[1 - i])
            torch.cuda.synchronize()
            for n in want[i]:
                assert torch.equal(got[i][n], want[i][n]), (turn, i, n)
                assert torch.equal(eager[n], want[1 - i][n]), (turn, i, n)


def test_rule_offsets_beyond_32_bits():
    """q, k, v and y of over 2^32 bytes: the last row equals the row alone."""
    B, T, H, K, V = 8200, 128, 16, 128, 128
    assert B * T * H * V * 2 > 2 ** 32
    small = inputs(1, T, H, H, K, V, BF16, norm=True, s0=False)
    big = {n: torch.zeros((B,) + small[n].shape[1:], device="cuda", dtype=small[n].dtype) for n in IN + ("dy",)}
    for n in big:
        big[n][-1] = small[n][0]
    big.update(s0=None, dsT=None)
    small["dsT"] = None
    a, b = run(big, norm=True), run(small, norm=True)
    for n in ("y",) + tuple("d" + m for m in IN):
        assert torch.equal(a[n][-1], b[n][0]), n
        assert not a[n][-2].any(), n
    assert torch.equal(a["sT"][-1], b["sT"][0])


# B, T, Hk, Hv, K, V, dtype, norm, s0, dsT, record
MANY = [
    (4, 130, 16, 32, 64, 64, BF16, True, True, True, True),     # 128 heads of 64 and more: the scans
    (8, 64, 16, 16, 64, 16, BF16, False, True, True, False),    # make their triangular factors themselves
    (3, 199, 15, 45, 64, 48, BF16, True, False, True, True),
    (2, 1, 64, 64, 64, 32, BF16, False, True, True, True),
    (4, 130, 16, 32, 64, 80, BF16, True, True, True, True),     # and not: wider values
    (11, 70, 3, 27, 128, 96, BF16, True, True, False, True),    # more workgroups than compute units
    (2, 90, 5, 10, 128, 256, F32, False, True, True, True),     # 16 slabs of 20 heads
    (17, 66, 1, 1, 64, 256, BF16, True, True, True, True),
]


@pytest.mark.parametrize("case", MANY, ids=["-".join(map(str, c)).replace("torch.", "") for c in MANY])
def test_rule_many_heads(case):
    test_rule(case)


@pytest.mark.parametrize("starts", PACKED[:4], ids=[str(i) for i in range(4)])
def test_rule_packed_many_heads(starts):
    """As test_rule_packed, with the factors made by the scans' workgroups."""
    T, H = starts[-1] + 9, 128
    d = inputs(1, T, 32, H, 64, 32, BF16, starts=starts, norm=True)
    for n in IN + ("dy",):
        d[n][:, :starts[0]] = float("nan")
        d[n][:, starts[-1]:] = float("nan")
    got = run(d, starts=starts, norm=True)
    inside = slice(starts[0], starts[-1])
    for n in ("y",) + tuple("d" + m for m in IN):   # what is outside is not written
        got[n] = got[n][:, inside]
    want = reference(d, starts=starts, norm=True)
    want = {n: w if n in ("sT", "ds0") else w[:, inside] for n, w in want.items()}
    check(got, want, f"many {starts}")


def test_rule_extreme_gates_many_heads():
    """test_rule_extreme_gates' gates and keys, in 128 heads."""
    d = inputs(1, 150, 128, 128, 64, 16, BF16, norm=True)
    g, be = d["g"], d["beta"]
    g[:, 10:30:4] = -float("inf")
    g[:, 70, 0] = -1e30
    g[:, 71, 0] = -200.0
    g[:, 90:128, 1] = 0.0
    be[:, 20:40] = 0.0
    be[:, 90:110] = 1.0
    d["k"][:, 80:128] = d["k"][:, 80:81]
    d["k"][:, 5] = 0
    d["q"][:, 6] = 0
    check(run(d, norm=True), reference(d, norm=True), "gates, many")


def test_rule_heads_do_not_leak():
    """inf and NaN in one head stay in it."""
    d = inputs(1, 100, 128, 128, 64, 64, BF16)
    clean = run(d)
    for n, x in (("v", float("inf")), ("q", float("nan")), ("dy", float("inf")), ("g", float("nan"))):
        d[n][:, 40, 77] = x
    got = run(d)
    for n in ("y",) + tuple("d" + m for m in IN):
        for part in (slice(0, 77), slice(78, 128)):
            assert torch.equal(got[n][:, :, part], clean[n][:, :, part]), n


def test_rule_scale_tensor_changed_in_place():
    """A scale given as a tensor is read at every call."""
    d = inputs(1, 20, 1, 1, 64, 16, F32)
    a, s = [d[n] for n in IN], torch.tensor(0.5)
    y0 = api.gdr_forward(*a, scale=s)[0]
    s.fill_(1.0)
    assert torch.equal(api.gdr_forward(*a, scale=s)[0], 2 * y0)


def test_rule_two_calls_at_once():
    """Calls on two streams with nothing between them, again and again."""
    d = [inputs(4, 150, 16, 32, 64, 64, BF16, seed=3), inputs(2, 200, 2, 4, 128, 64, F32, seed=4)]
    want = [run(x) for x in d]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in d]
    got = [[run(x, stream=s) for _ in range(3)] for x, s in zip(d, streams)]
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        for one in g:
            for n in w:
                assert torch.equal(one[n], w[n]), n


def test_rule_many_heads_captured():
    """A captured forward and backward whose workgroups make the factors."""
    d = inputs(4, 100, 16, 32, 64, 64, BF16, seed=9)
    want, g = run(d), torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=side):
        got = run(d)
    for _ in range(3):
        for x in got.values():
            x.zero_()
        g.replay()
        eager = run(d)
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(got[n], want[n]) and torch.equal(eager[n], want[n]), n


# ---------------------------------------------------------------------- decode

@pytest.mark.parametrize("B,T,Hk,Hv,K,V,dt,norm", [
    (1, 1, 1, 1, 64, 16, F32, False), (3, 1, 2, 4, 128, 128, BF16, True), (5, 4, 1, 3, 64, 80, BF16, True),
    (2, 3, 2, 2, 128, 48, F32, True), (70, 1, 1, 1, 64, 64, F32, False), (2, 9, 1, 1, 64, 256, BF16, False)])
def test_decode(B, T, Hk, Hv, K, V, dt, norm):
    print(f"decode {B} {T} {Hk} {Hv} {K} {V} {dt} {norm}", flush=True)
    d = inputs(B, T, Hk, Hv, K, V, dt, norm=norm)
    pool = torch.randn(B + 4, Hv, V, K, device="cuda")
    slots = torch.randperm(B + 4, device="cuda")[:B].to(torch.int32)
    pool[slots.long()] = d["s0"]
    before = pool.clone()
    y = api.gdr_decode(*(d[n] for n in IN), pool, slots, norm_qk=norm)
    want = R.rule(*(d[n] for n in IN), d["s0"], norm_qk=norm)
    check(dict(y=y, sT=pool[slots.long()]), want, "decode")
    rest = torch.ones(B + 4, dtype=torch.bool, device="cuda")
    rest[slots.long()] = False
    assert torch.equal(pool[rest], before[rest])
    # in place over the first B states, and against the chunked form
    own = d["s0"].clone()
    y2 = api.gdr_decode(*(d[n] for n in IN), own, norm_qk=norm)
    assert torch.equal(y2, y) and torch.equal(own, pool[slots.long()])


def test_decode_skipped_rows():
    """Slots outside the pool, and a slot named again."""
    B, pool = 7, 6
    d = inputs(B, 2, 1, 2, 64, 32, F32)
    state = torch.randn(pool, 2, 32, 64, device="cuda")
    slots = torch.tensor([2, -1, 5, 2, 6, 0, 5], dtype=torch.int32, device="cuda")
    live = [0, 2, 5]
    before, y = state.clone(), torch.full((B, 2, 2, 32), 7.0, device="cuda")
    api.gdr_decode(*(d[n] for n in IN), state, slots, out=y)
    at = slots[live].long()
    want = R.rule(*(d[n][live] for n in IN), before[at])
    check(dict(y=y[live], sT=state[at]), want, "skipped")
    skipped = [i for i in range(B) if i not in live]
    assert (y[skipped] == 7).all()
    for i in (1, 3, 4):
        assert torch.equal(state[i], before[i])


def test_decode_continues_prefill():
    """Tokens one by one from the chunked form's state, replayed as a graph."""
    T0, T1 = 70, 5
    d = inputs(2, T0 + T1, 1, 2, 64, 48, BF16, norm=True)
    want = R.rule(*(d[n] for n in IN), d["s0"], norm_qk=True)
    state = api.gdr_forward(*(d[n][:, :T0].contiguous() for n in IN), d["s0"], norm_qk=True)[1]
    step = [d[n][:, T0:T0 + 1].clone() for n in IN]
    start = state.clone()
    api.gdr_decode(*step, state, norm_qk=True)   # warm
    state.copy_(start)
    gr = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(gr):
        y = api.gdr_decode(*step, state, norm_qk=True)
    ys = []
    for t in range(T1):
        for x, n in zip(step, IN):
            x.copy_(d[n][:, T0 + t:T0 + t + 1])
        gr.replay()
        ys.append(y.clone())
    check(dict(y=torch.cat(ys, 1)), dict(y=want["y"][:, T0:]), "decode")
    check(dict(sT=state), dict(sT=want["sT"]), "decode")


def test_decode_pool_beyond_32_bits():
    Hv, V, K = 32, 128, 128
    n = 2 ** 32 // (Hv * V * K * 4) + 3
    d = inputs(1, 1, 16, Hv, K, V, BF16, norm=True)
    pool = torch.zeros(n, Hv, V, K, device="cuda")
    pool[-1] = d["s0"][0]
    slots = torch.tensor([n - 1], dtype=torch.int32, device="cuda")
    y = api.gdr_decode(*(d[m] for m in IN), pool, slots, norm_qk=True)
    own = d["s0"].clone()
    assert torch.equal(api.gdr_decode(*(d[m] for m in IN), own, norm_qk=True), y)
    assert torch.equal(own[0], pool[-1]) and not pool[0].any()


# ----------------------------------------------------------------------- norms

@pytest.mark.parametrize("rows,H,N,heads,dt", [
    (1, 1, 16, False, F32), (3, 5, 32, True, BF16), (7, 2, 64, False, BF16), (130, 3, 64, True, F32),
    (33, 7, 128, True, BF16), (5, 3, 256, False, F32), (2000, 3, 64, False, BF16)])
def test_epilogue(rows, H, N, heads, dt):
    print(f"epilogue {rows} {H} {N} {heads} {dt}", flush=True)
    gen = torch.Generator().manual_seed(2)
    y, g, dz = (torch.randn(1, rows, H, N, generator=gen).to(dt).cuda() for _ in range(3))
    w = torch.randn(H if heads else 1, N, generator=gen).cuda()
    got = dict(api.gdr_epilogue_backward(dz, y, g, w), z=api.gdr_epilogue_forward(y, g, w))
    check(got, R.epilogue(y, g, w, dz), "epilogue")
    again = api.gdr_epilogue_backward(dz, y, g, w)
    for n in again:
        assert torch.equal(again[n], got[n])


def test_epilogue_extremes():
    """Rows of zeros, gates that saturate (exp overflows), no rows at all."""
    y, g = torch.randn(1, 4, 1, 64, device="cuda"), torch.randn(1, 4, 1, 64, device="cuda")
    y[:, 1], g[:, 2], g[:, 3] = 0, 200.0, -200.0
    w = torch.ones(1, 64, device="cuda")
    dz = torch.randn_like(y)
    got = dict(api.gdr_epilogue_backward(dz, y, g, w), z=api.gdr_epilogue_forward(y, g, w))
    check(got, R.epilogue(y, g, w, dz), "extremes")
    e = torch.empty(1, 0, 3, 64, device="cuda")
    assert api.gdr_epilogue_forward(e, e, w).shape == e.shape
    assert not api.gdr_epilogue_backward(e, e, e, w)["dw"].any()


@pytest.mark.parametrize("rows,D,scaled,dt", [
    (1, 1, True, F32), (3, 7, False, BF16), (5, 64, True, BF16), (9, 511, True, F32), (130, 1000, False, F32),
    (6, 1025, True, BF16), (3, 2048, True, F32), (1500, 776, True, BF16), (4, 4097, False, BF16),
    (3, 8200, True, F32), (2, 16384, True, BF16), (2, 16383, True, F32)])
def test_residual_norm(rows, D, scaled, dt):
    print(f"norm {rows} {D} {scaled} {dt}", flush=True)
    gen = torch.Generator().manual_seed(3)
    x, y, dh, dx = (torch.randn(rows, D, generator=gen).to(dt).cuda() for _ in range(4))
    w, s = (torch.randn(D, generator=gen).cuda() for _ in range(2))
    s = s if scaled else None
    xo, h = api.residual_norm_forward(x, y, w, s)
    check(dict(x_out=xo, h=h), R.residual_norm(x, y, w, s), "norm")
    args = (dh, dx, xo, w) + ((y, s) if scaled else ())
    got = api.residual_norm_backward(*args)
    check(got, R.residual_norm_backward(*args), "norm")
    # in place, and without the branch or the gradient of the stream
    x2, dx2 = x.clone(), dx.clone()
    xo2, h2 = api.residual_norm_forward(x2, y, w, s, out=(x2, None))
    assert xo2 is x2 and torch.equal(x2, xo) and torch.equal(h2, h)
    got2 = api.residual_norm_backward(dh, dx2, *args[2:], out=dict(dx=dx2))
    for n in got:
        assert got[n] is None or torch.equal(got2[n], got[n]), n
    xo3, h3 = api.residual_norm_forward(x, None, w)
    assert torch.equal(xo3, x)
    check(dict(h=h3), R.residual_norm(x, None, w), "plain")
    # dx = r (dh w - xn mean(dh w xn)), xn^2 <= D: with one entry to a row,
    # xn^2 = 1 - eps / x^2 and the two terms, of size r |dh w| each, cancel but
    # for eps / x^2 = 1e-6 of them.  Each term carries roundings of 2^-24 of itself.
    xd = xo.cpu().double()
    # (dy and dscale are dx times scale and y.)
    term = dh.cpu().double() * w.cpu().double() / (xd.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    check(api.residual_norm_backward(dh, None, *args[2:]), R.residual_norm_backward(dh, None, *args[2:]), "no dx",
          dict(dx=float(term.norm()), dy=0.0 if s is None else float((term * s.cpu().double()).norm()),
               dscale=float((term * y.cpu().double()).abs().sum(0).norm())))


@pytest.mark.parametrize("rows,D,scaled,dt", [
    (2100, 8200, True, BF16), (1030, 16384, True, F32), (2050, 4096, True, BF16), (1100, 8192, False, BF16)])
def test_residual_norm_more_rows_than_workgroups(rows, D, scaled, dt):
    test_residual_norm(rows, D, scaled, dt)


def test_residual_norm_captured_and_empty():
    x, y = (torch.randn(70, 300, device="cuda") for _ in range(2))
    w, s = (torch.randn(300, device="cuda") for _ in range(2))
    want = api.residual_norm_backward(y, x, x, w, y, s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=side):
        got = api.residual_norm_backward(y, x, x, w, y, s)
    for _ in range(3):
        got["dw"].zero_()
        gr.replay()
        eager = api.residual_norm_backward(y, x, x, w, y, s)
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(got[n], want[n]) and torch.equal(eager[n], want[n]), n
    e = torch.empty(0, 300, device="cuda")
    assert api.residual_norm_forward(e, e, w, s)[1].shape == e.shape
    g = api.residual_norm_backward(e, e, e, w, e, s)
    assert not g["dw"].any() and not g["dscale"].any()


# --------------------------------------------------------------------- together

def test_block_and_its_gradients():
    """A block as a model has it: residual norm, projections, the rule, its
    epilogue, the output projection, the next residual norm; the gradients
    chained back through the calls, against autograd in 64 bits."""
    B, T, D, Hk, Hv, K, V = 2, 90, 96, 1, 2, 64, 32
    gen = torch.Generator().manual_seed(8)

    def rn(*s):
        return torch.randn(s, generator=gen)

    W = {n: rn(D, m) / D ** 0.5 for n, m in (("q", Hk * K), ("k", Hk * K), ("v", Hv * V), ("z", Hv * V))}
    W["o"] = rn(Hv * V, D) / (Hv * V) ** 0.5
    x, y0, dh = rn(B, T, D), rn(B, T, D), rn(B, T, D)
    w1, w2, sc, wn = 1 + 0.1 * rn(D), 1 + 0.1 * rn(D), rn(D), 1 + 0.1 * rn(1, V)
    g, be = -rn(B, T, Hv).abs(), torch.sigmoid(rn(B, T, Hv))
    names = ("x", "y0", "w1", "w2", "sc", "wn", "g", "be")
    leaf = {n: t.double().requires_grad_() for n, t in zip(names, (x, y0, w1, w2, sc, wn, g, be))}
    Wd = {n: t.double() for n, t in W.items()}

    def rms(t, w, n):
        return t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-6) * w

    x1 = leaf["x"] + leaf["sc"] * leaf["y0"]
    h1 = rms(x1, leaf["w1"], D)
    q, k = ((h1 @ Wd[n]).view(B, T, Hk, K) for n in ("q", "k"))
    q, k = (t / torch.sqrt((t * t).sum(-1, keepdim=True) + 1e-6) for t in (q, k))
    v = (h1 @ Wd["v"]).view(B, T, Hv, V)
    S = torch.zeros(B, Hv, V, K, dtype=torch.float64)
    ys = []
    for t in range(T):
        kt, qt = (u[:, t].repeat_interleave(Hv // Hk, 1) for u in (k, q))
        S = S * torch.exp(leaf["g"][:, t])[..., None, None]
        u = leaf["be"][:, t][..., None] * (v[:, t] - (S * kt[..., None, :]).sum(-1))
        S = S + u[..., None] * kt[..., None, :]
        ys.append((S * qt[..., None, :]).sum(-1) * K ** -0.5)
    o = torch.stack(ys, 1)
    gate = (h1 @ Wd["z"]).view(B, T, Hv, V)
    z = rms(o, leaf["wn"], V) * torch.nn.functional.silu(gate)
    x2 = x1 + z.reshape(B, T, -1) @ Wd["o"]
    h2 = rms(x2, leaf["w2"], D)
    want = dict(zip(names, torch.autograd.grad((h2 * dh.double()).sum(), [leaf[n] for n in names])))

    c = {n: t.cuda() for n, t in zip(names, (x, y0, w1, w2, sc, wn, g, be))}
    Wc = {n: t.cuda() for n, t in W.items()}
    gx1, gh1 = api.residual_norm_forward(c["x"], c["y0"], c["w1"], c["sc"])
    gq, gk = ((gh1 @ Wc[n]).view(B, T, Hk, K) for n in ("q", "k"))
    gv, gg = ((gh1 @ Wc[n]).view(B, T, Hv, V) for n in ("v", "z"))
    go, _, ck = api.gdr_forward(gq, gk, gv, c["g"], c["be"], norm_qk=True, want_ckpt=True, want_sT=False)
    gz = api.gdr_epilogue_forward(go, gg, c["wn"])
    gx2, gh2 = api.residual_norm_forward(gx1, (gz.view(B, T, -1) @ Wc["o"]), c["w2"])
    b2 = api.residual_norm_backward(dh.cuda(), None, gx2, c["w2"])
    ep = api.gdr_epilogue_backward((b2["dx"] @ Wc["o"].t().contiguous()).view(B, T, Hv, V), go, gg, c["wn"])
    r = api.gdr_backward(gq, gk, gv, c["g"], c["be"], ep["dy"], None, None, ck, norm_qk=True, want_ds0=False)
    gh = sum(t.reshape(B, T, -1) @ Wc[n].t().contiguous()
             for n, t in (("q", r["dq"]), ("k", r["dk"]), ("v", r["dv"]), ("z", ep["dgate"])))
    b1 = api.residual_norm_backward(gh, b2["dx"], gx1, c["w1"], c["y0"], c["sc"])
    got = dict(x=b1["dx"], y0=b1["dy"], w1=b1["dw"], w2=b2["dw"], sc=b1["dscale"], wn=ep["dw"], g=r["dg"],
               be=r["dbeta"])
    check(dict(h=gh2), dict(h=h2.detach()), "block")
    check(got, want, "block")
