"""Softmax attention, its norm and its cache at sizes that take them through paths
which small shapes do not reach: dies that take their units in turns, two heads at a
time and angles formed again in the norm, the search for a packed token's row over
several levels, short rows in wide tables; MI355X only.  Bars as in
test_attention_gpu."""
import math

import pytest
import torch

import oracle.attention as R
from linear_attention_rnn_wkv7_amd import api
from test_attention_gpu import BF16, E4M3, F32, HALF_STEP, check, inputs, qk_inputs, qk_run, run
from test_attention_gpu import test_cache as check_cache
from test_attention_gpu import test_decode as check_decode

pytestmark = pytest.mark.gpu

TURNS = [
    # B, T, Hq, Hk, D, dtype: a die has more units than it takes at a time, and the last
    # time fewer
    (17, 1025, 8, 8, 128, F32), (33, 1025, 8, 8, 64, BF16), (17, 1100, 16, 8, 128, BF16),
]


@pytest.mark.parametrize("case", TURNS, ids=["-".join(map(str, c)).replace("torch.", "") for c in TURNS])
def test_units_in_turns(case):
    """Rows that differ by powers of two in v and dy: so do, exactly, y and the gradients;
    the first is compared with the oracle."""
    B, T, Hq, Hk, D, dt = case
    one = inputs(1, T, Hq, Hk, D, dt, seed=100)
    row = torch.arange(B, device="cuda").view(B, 1, 1, 1)
    by = {"v": torch.exp2((row % 7).float()), "dy": torch.exp2(-(row % 5).float())}
    d = {n: (x.float() * by.get(n, 1.0)).to(dt).expand(B, -1, -1, -1).contiguous() for n, x in one.items()}
    got = run(d)
    check({n: x[:1] for n, x in got.items()}, R.attention(*(one[n] for n in ("q", "k", "v", "dy"))), str(case), D=D, T=T)
    both = by["v"] * by["dy"]
    for n, f in (("y", by["v"]), ("dq", both), ("dk", both), ("dv", by["dy"])):
        assert torch.equal(got[n].float(), got[n][:1].float() * f), n
    assert torch.equal(got["lse"], got["lse"][:1].expand(B, -1, -1))


def qk_reference(d, step=2048, **kw):
    """oracle.attention's qk_norm of one long row, some tokens at a time."""
    T, out, sums = d["q"].shape[1], [], {}
    for lo in range(0, T, step):
        s = {n: x if x is None or n in ("wq", "wk", "theta") else x[:, lo:lo + step] for n, x in d.items()}
        w = R.qk_norm(*(s[n] for n in ("q", "k", "wq", "wk", "theta", "positions", "dq", "dk")), **kw)
        out.append({n: w[n] for n in ("q", "k", "dq", "dk")})
        for n in ("dwq", "dwk"):
            sums[n] = sums.get(n, 0) + w[n]
            sums[n + "_2"] = sums.get(n + "_2", 0) + w[n + "_2"] ** 2
    whole = {n: torch.cat([w[n] for w in out], 1) for n in ("q", "k", "dq", "dk")}
    return dict(whole, **{n: x.sqrt() if n.endswith("_2") else x for n, x in sums.items()})


QK = [
    # T, Hq, Hk, D, R, dtype.  A step takes 64 (of 128: 32) heads of a workgroup's tokens
    (3, 40, 17, 64, 64, F32), (3, 40, 17, 128, 64, F32), (3, 40, 17, 64, 32, BF16), (3, 40, 17, 128, 128, BF16),
    (1, 65, 33, 64, 48, F32), (2, 100, 31, 128, 96, F32), (5, 33, 129, 64, 64, BF16),
    # angles are in LDS for 16 tokens at a time
    (33000, 3, 1, 64, 32, F32), (33000, 3, 1, 128, 64, F32), (33000, 5, 2, 64, 64, BF16), (17000, 3, 2, 128, 32, BF16),
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", QK, ids=["-".join(map(str, c)).replace("torch.", "") for c in QK])
def test_qk_norm_steps(case, interleaved):
    """fp32 and bf16 as in test_attention_gpu.qk_check; a second call gives the same bits."""
    T, Hq, Hk, D, R_, dt = case
    d = qk_inputs(1, T, Hq, Hk, D, R_, dt, seed=101)
    got, again = (qk_run(d, interleaved=interleaved) for _ in range(2))
    for n in got:
        assert torch.equal(got[n], again[n]), n
    want = qk_reference(d, interleaved=interleaved)
    for n in ("q", "k", "dq", "dk"):
        g, w = got[n].cpu().double(), want[n]
        most = HALF_STEP[dt] * w.abs() + (4 * 128 ** 0.5 * 2.0 ** -24 + 2.0 ** -20) * w.norm(dim=-1, keepdim=True) + 1e-30
        err = (g - w).abs()
        assert (err <= most).all(), (case, n, float((err / most).max()))
    for n, H in (("dwq", Hq), ("dwk", Hk)):
        most = ((T * H) ** 0.5 + 16) * 2.0 ** -22 * want[n + "_2"] + 1e-30
        assert ((got[n].cpu().double() - want[n]).abs() <= most).all(), (case, n)


def many_rows(rows, first, seed):
    """Starts of so many short sequences, empty ones at the borders of the search's ranges."""
    gen = torch.Generator().manual_seed(seed)
    n = torch.randint(0, 6, (rows,), generator=gen)
    for i in (0, 7, 8, 15, 16, 63, 64, 127, 255, 256, rows - 1):
        if i < rows:
            n[i] = 0 if i % 2 else 3
    return [first] + (first + n.cumsum(0)).tolist(), (n + torch.randint(0, 20, (rows,), generator=gen)).tolist()


@pytest.mark.parametrize("rows", [8, 9, 16, 17, 64, 65, 257, 700])
@pytest.mark.parametrize("D, dt, kind", [(64, BF16, BF16), (128, BF16, BF16), (64, F32, E4M3), (128, BF16, E4M3)])
def test_cache_of_many_rows(rows, D, dt, kind):
    """A packed token's row is found by 8 or 16 lanes (heads of 64 or 128), level by level."""
    starts, lens = many_rows(rows, 3, rows)
    check_cache((rows, starts, 2, 16, 1 + rows % 2, D, dt, kind, lens))


SHORT = [
    (2, 1, 8, 2, 64, 64, 300, BF16, BF16, [70, 1]), (3, 1, 4, 1, 128, 16, 500, BF16, E4M3, [33, 500, 0]),
    (2, 3, 4, 2, 64, 32, 400, F32, F32, [2, 1000]), (1, 1, 2, 2, 128, 256, 64, F32, E4M3, [40]),
]


@pytest.mark.parametrize("case", SHORT, ids=["-".join(map(str, c[:9])).replace("torch.", "") for c in SHORT])
def test_decode_short_rows_in_wide_tables(case):
    """Parts follow the table: here most of them have nothing, or one step."""
    assert api.attn_decode_workspace_bytes(*case[:5], 1, case[5], case[6]) > 0
    check_decode(case)


def test_largest_scale():
    """2^127: scores of 0 weigh all keys alike."""
    q, k = torch.zeros(1, 5, 2, 64, device="cuda"), torch.randn(1, 5, 1, 64, device="cuda")
    v = torch.arange(5.0, device="cuda").view(1, 5, 1, 1).expand(1, 5, 1, 64).contiguous()
    y, lse, _ = api.attn_forward(q, k, v, scale=2.0 ** 127, want_lse=True)
    assert torch.equal(y, (torch.arange(5.0, device="cuda") / 2).view(1, 5, 1, 1).expand_as(y))
    assert float((lse - torch.log(torch.arange(1.0, 6.0, device="cuda")).view(1, 5, 1)).abs().max()) <= 2.0 ** -22 * math.log(5)
    with pytest.raises(RuntimeError, match="invalid"):
        api.attn_forward(q, k, v, scale=3e38)
