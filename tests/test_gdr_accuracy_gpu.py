"""Accuracy of the gated delta rule where a result is small beside what it is
made of, MI355X only: reads of an overwritten key, gradients of fast decays."""
import pytest
import torch

import oracle.gdr as R
from linear_attention_rnn_wkv7_amd import api
from test_gdr_gpu import BF16, F32, HALF_STEP

pytestmark = pytest.mark.gpu


# B, T, Hk, Hv, K, V, dtype: the scan finds its triangular factors in memory,
# makes them itself (128 heads and more of 64), has keys of 128
SHAPES = [(1, 100, 1, 2, 64, 32, BF16), (2, 100, 64, 64, 64, 48, BF16), (1, 140, 2, 2, 128, 64, BF16),
          (1, 100, 1, 2, 64, 32, F32)]


@pytest.mark.parametrize("case", SHAPES, ids=["-".join(map(str, c)).replace("torch.", "") for c in SHAPES])
def test_read_of_an_overwritten_key(case):
    """Unit keys that are columns of the identity, beta 1, no decay: token i
    replaces column i mod K of a state 4096 times as large as its values, and
    reads a column that an earlier token of its chunk, itself or no token has
    replaced:
        y = s0 + sum of (v - what stood there)
    Every product has one factor 1 and every sum one or two terms besides
    zeros, in three parts at most.  Between s0 and y stand six operands of at
    most 24 bits or more (s0 twice, the difference twice, the replaced column
    once a chunk on the way) and at most ten sums, each off by 2^-24 of s0:
    16 * 2^-24 |s0|, besides the half step of y's type."""
    B, T, Hk, Hv, K, V, dt = case
    print(f"case {case}", flush=True)
    gen = torch.Generator().manual_seed(6)
    s0 = 4096 * torch.randn(B, Hv, V, K, generator=gen)
    v = torch.randn(B, T, Hv, V, generator=gen).to(dt)
    t = torch.arange(T)
    eye = torch.eye(K)
    k = eye[t % K][None, :, None, :].expand(B, T, Hk, K).contiguous().to(dt)
    q = eye[(37 * t + 11) % K][None, :, None, :].expand(B, T, Hk, K).contiguous().to(dt)
    q[:, ::3] = k[:, ::3]
    g, beta = torch.zeros(B, T, Hv), torch.ones(B, T, Hv)
    y = api.gdr_forward(*(x.cuda() for x in (q, k, v, g, beta, s0)), scale=1.0)[0].cpu().double()
    want = R.rule(q, k, v, g, beta, s0, scale=1.0)["y"]
    column = q.double()[:, :, 0].argmax(-1)                      # [B, T]
    old = torch.stack([s0[b][:, :, column[b]].permute(2, 0, 1) for b in range(B)]).abs().double()
    small = want.abs() < 64                                      # the replaced ones
    assert small.float().mean() > 0.3 and (old / want.abs())[small].median() > 1000
    err, bar = (y - want).abs(), HALF_STEP[dt] * want.abs() + 16 * 2.0 ** -24 * old
    print(f"overwritten {case}: worst {float((err / bar).max()):.3f} of the bar", flush=True)
    assert (err <= bar).all(), float((err / bar).max())
