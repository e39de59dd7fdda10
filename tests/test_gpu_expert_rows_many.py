"""Expert rows of very many short rows: every row is reached."""
import pytest
import torch

import sparse_selection_primitive_b200 as L

pytestmark = pytest.mark.gpu


def test_rows_past_the_largest_wave(cuda_device):
    """1.3e9 rows of one element (2^20 blocks an SM, of 8 rows each, hold 1.24e9): all values are
    small whole numbers or quarters, so the results are exact."""
    T = 1_300_000_000
    at = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = at.flip(0).view(T, 1)                   # row t lies at place T - 1 - t
    offsets = torch.tensor([0, T - 5], dtype=torch.int32, device="cuda")  # the last five places: dropped
    plan = L.ExpertPlan(offsets, slots, slots.view(-1))
    dout = (at % 3 - 1).to(torch.bfloat16).view(T, 1)
    w = (at % 5).float().mul_(0.25).view(T, 1).requires_grad_(True)
    y = (at % 7).to(torch.bfloat16).view(T, 1).requires_grad_(True)
    out = L.expert_combine(y, w, plan)
    dy, dw = torch.autograd.grad(out, (y, w), dout)
    del at, slots
    step = 1 << 27
    for a in range(0, T, step):
        b = min(T, a + step)
        t = torch.arange(a, b, device="cuda")
        place = T - 1 - t
        live = place < T - 5
        g, wt, yt = (t % 3 - 1).float(), (t % 5).float() * 0.25, (place % 7).float()
        assert torch.equal(out[a:b, 0].float(), torch.where(live, wt * yt, 0.0))
        assert torch.equal(dw[a:b, 0], torch.where(live, g * yt, 0.0))
        back = torch.where(live, wt * g, 0.0).flip(0)
        assert torch.equal(dy[T - b:T - a, 0].float(), back)
    del out, dy, dw
    x = dout[:, :]
    xs = L.expert_gather(x, plan)
    for a in range(0, T, step):
        b = min(T, a + step)
        t = torch.arange(a, b, device="cuda")
        got = xs[T - b:T - a, 0].flip(0).float()
        assert torch.equal(got, torch.where(T - 1 - t < T - 5, (t % 3 - 1).float(), 0.0))
