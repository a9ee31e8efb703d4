"""The gradient of the gated delta rule's log decay, head by head, MI355X
only.  It carries the decay as a factor, so in a head that forgets fast it is
small beside the products it is made of.

Bar.  That of tests/test_gdr_gpu.py for the sums, 8.1e-6 in the 2-norm, but
of each head by itself; and the decay between two tokens is 2 to the power of
a difference d of log sums, whose roundings, 2^-24 |d| twice, count ln 2 of
that: |d| is |g| log2(e) for the terms that matter."""
import pytest
import torch

import oracle.gdr as R
from test_gdr_gpu import BF16, F32, IN, REL, inputs, run

pytestmark = pytest.mark.gpu
RATES = (-0.01, -0.1, -1.0, -4.0, -10.0, -16.0, -30.0, -60.0)

# B, T, Hk, Hv, K, V, dtype, norm
CASES = [(1, 200, 8, 8, 64, 64, F32, False), (1, 200, 4, 8, 64, 48, BF16, True), (1, 150, 8, 8, 128, 64, BF16, False),
         (1, 150, 4, 8, 128, 80, F32, True), (1, 100, 128, 128, 64, 32, BF16, True), (2, 1100, 1, 2, 64, 16, F32, False)]


@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c)).replace("torch.", "") for c in CASES])
def test_decay_gradient_of_each_head(case):
    B, T, Hk, Hv, K, V, dt, norm = case
    print(f"case {case}", flush=True)
    d = inputs(B, T, Hk, Hv, K, V, dt, norm=norm, seed=11)
    rate = torch.tensor([RATES[(b * Hv + h) % 8] for b in range(B) for h in range(Hv)]).view(B, 1, Hv)
    d["g"] = (rate * (0.8 + 0.4 * torch.rand(B, T, Hv, generator=torch.Generator().manual_seed(2)))).cuda()
    got = run(d, norm=norm)["dg"].cpu().double()
    want = R.rule(*(d[n] for n in IN), d["s0"], d["dy"], d["dsT"], norm_qk=norm)["dg"]
    worst = 0.0
    for b in range(B):
        for h in range(Hv):
            w, r = want[b, :, h], float(rate[b, 0, h])
            bar = REL + 2 * 1.2 * abs(r) * 2.0 ** -24
            rel = float((got[b, :, h] - w).norm() / w.norm())
            worst = max(worst, rel / bar)
            if Hv <= 8:
                print(f"{case} g {r}: dg {rel:.2e} (bar {bar:.2e})", flush=True)
    assert worst <= 1, worst


@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c)).replace("torch.", "") for c in CASES])
def test_decay_gradient_of_a_forgotten_state(case):
    """Exactly zero at g <= -200, -inf among them."""
    B, T, Hk, Hv, K, V, dt, norm = case
    print(f"case {case}", flush=True)
    d = inputs(B, T, Hk, Hv, K, V, dt, norm=norm, seed=12)
    d["g"][:, 3::7] = -200.0
    d["g"][:, 5::11] = -float("inf")
    d["g"][:, 64:66] = -1e30
    dg = run(d, norm=norm)["dg"]
    gone = d["g"] <= -200
    assert (dg[gone] == 0).all(), float(dg[gone].abs().max())
    assert (dg[~gone] != 0).float().mean() > 0.9
