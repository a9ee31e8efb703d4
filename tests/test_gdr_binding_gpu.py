"""What the torch binding of the gated delta rule and the norms takes, MI355X
only."""
import pytest
import torch

from linear_attention_rnn_wkv7_amd import api
from test_gdr_gpu import BF16, F32, IN, inputs

pytestmark = pytest.mark.gpu


def _off(t, n=1):
    """The same values, `n` elements off an allocation's start."""
    big = torch.empty(t.numel() + n, device=t.device, dtype=t.dtype)
    big[n:] = t.reshape(-1)
    out = big[n:].view(t.shape)
    assert out.data_ptr() % 16 != 0 and out.is_contiguous()
    return out


@pytest.mark.parametrize("n", [1, 2, 3])
def test_slices_of_slots_starts_and_gates(n):
    """Slots, starts, g and beta that begin anywhere, as slices of a batch's do."""
    starts = [0, 3, 40, 75]
    d = inputs(1, 75, 1, 3, 64, 32, BF16, starts=starts)
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")
    a = [d[m] for m in IN]
    b = a[:3] + [_off(a[3], n), _off(a[4], n)]
    want = api.gdr_forward(*a, d["s0"], seq_starts=st, want_ckpt=True)
    got = api.gdr_forward(*b, d["s0"], seq_starts=_off(st, n), want_ckpt=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    gw = api.gdr_backward(*a, d["dy"], d["s0"], d["dsT"], want[2], seq_starts=st)
    gg = api.gdr_backward(*b, d["dy"], d["s0"], d["dsT"], got[2], seq_starts=_off(st, n))
    for m in gw:
        assert torch.equal(gg[m], gw[m]), m
    d = inputs(5, 1, 1, 3, 64, 32, F32)
    pool = torch.randn(8, 3, 32, 64, device="cuda")
    slots = torch.tensor([7, 2, 0, 5, 1], dtype=torch.int32, device="cuda")
    p0, p1 = pool.clone(), pool.clone()
    y0 = api.gdr_decode(*(d[m] for m in IN), p0, slots)
    y1 = api.gdr_decode(*(d[m] for m in IN[:3]), _off(d["g"], n), _off(d["beta"], n), p1, _off(slots, n))
    assert torch.equal(y0, y1) and torch.equal(p0, p1)


def test_slice_of_slots_captured():
    """A replay reads the slice as it then is."""
    d = inputs(3, 1, 1, 2, 64, 32, F32)
    pool = torch.randn(8, 2, 32, 64, device="cuda")
    every = torch.zeros(9, dtype=torch.int32, device="cuda")
    slots = every[1:4]
    assert slots.data_ptr() % 16 != 0
    slots.copy_(torch.tensor([0, 1, 2]))
    state, a = pool.clone(), [d[m] for m in IN]
    api.gdr_decode(*a, state, slots)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        y = api.gdr_decode(*a, state, slots)
    for turn in ([5, 1, 0], [2, 7, 3], [4, 4, 6], [0, 1, 2]):
        state.copy_(pool)
        slots.copy_(torch.tensor(turn))
        y.fill_(7.0)
        gr.replay()
        eager, out = pool.clone(), torch.full_like(y, 7.0)
        api.gdr_decode(*a, eager, torch.tensor(turn, dtype=torch.int32, device="cuda"), out=out)
        torch.cuda.synchronize()
        assert torch.equal(state, eager) and torch.equal(y, out), turn
