"""The norms around a recurrence with more rows than one launch has threads
for, MI355X only."""
import pytest
import torch

from linear_attention_rnn_wkv7_amd import api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,D,dt", [((1 << 22) + 5, 8, torch.bfloat16), ((1 << 26) + 37, 1, torch.bfloat16),
                                       ((1 << 22) + 5, 1030, torch.bfloat16)])
def test_residual_norm_more_rows_than_a_launch(rows, D, dt):
    """Rows of zeros and, across the launches' borders and at the end, others:
    as those alone."""
    print(f"norm {rows} {D}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(4)
    n = 100
    at = torch.cat([torch.arange(0, n), torch.arange((1 << 22) - n, (1 << 22) + 3), torch.arange(rows - n, rows)]).unique()
    at = torch.cat([at, torch.arange(min(rows, 1 << 26) - n, min(rows, 1 << 26))]).unique().cuda()
    small = [torch.randn(len(at), D, generator=gen, device="cuda").to(dt) for _ in range(3)]
    big = [torch.zeros(rows, D, device="cuda", dtype=dt) for _ in range(3)]
    for b, s in zip(big, small):
        b[at] = s
    w, sc = (torch.randn(D, generator=gen, device="cuda") for _ in range(2))
    xo, h = api.residual_norm_forward(big[0], big[1], w, sc)
    xs, hs = api.residual_norm_forward(small[0], small[1], w, sc)
    assert torch.equal(xo[at], xs) and torch.equal(h[at], hs)
    assert int((h != 0).any(1).sum()) <= len(at)
    del h
    want = api.residual_norm_backward(small[2], None, xs, w, small[1], sc)
    got = api.residual_norm_backward(big[2], None, xo, w, big[1], sc)
    for name in ("dx", "dy"):
        assert torch.equal(got[name][at], want[name]), name
    for name in ("dw", "dscale"):
        # the same few hundred terms, added up in another order: sqrt(400) steps of
        # 2^-24 of their 2-norm's size, 16 times that for a single sum
        terms = (len(at) ** 0.5) * float(want[name].abs().max()) + float(want[name].abs().sum() / D)
        assert float((got[name] - want[name]).abs().max()) <= 16 * 20 * 2.0 ** -24 * terms, name


@pytest.mark.parametrize("heads", [False, True])
def test_epilogue_more_rows_than_a_launch(heads):
    """2^29 heads of 16 and more, as those at the end alone."""
    H, N = 3, 16
    rows = (1 << 29) // H + 50
    gen = torch.Generator(device="cuda").manual_seed(5)
    small = [torch.randn(1, 40, H, N, generator=gen, device="cuda").bfloat16() for _ in range(2)]
    y, gate = (torch.zeros(1, rows, H, N, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    y[:, -40:], gate[:, -40:] = small
    w = torch.randn(H if heads else 1, N, generator=gen, device="cuda")
    z = api.gdr_epilogue_forward(y, gate, w)
    assert torch.equal(z[:, -40:], api.gdr_epilogue_forward(*small, w))
    assert not z[:, -80:-40].any()
