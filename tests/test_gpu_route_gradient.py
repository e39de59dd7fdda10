"""The routing gradient where one weight dominates, against the formula in 64 bits.

Tolerances, relative to each element's own sum of magnitudes: a renormalised or softmax
score is off by (2 |l - m| + 52) units of 2^-24 (the subtraction, the exponential's argument,
the sums), a sum over k by k + 4 more; four factors of that kind at most.  A sum of
differences, sum_j w_j (u_i - u_j), may be formed from two parts that are 2 k + 1 times its
magnitudes together, with three roundings each."""
import numpy as np
import pytest
import torch

import sparse_selection_primitive_b200 as L
from tests import select_reference as R

pytestmark = pytest.mark.gpu


def expected(l, idx, u, score, renormalize, scale):
    """(gradient, sum of magnitudes) of one row in float64."""
    s = np.exp(l - l.max()) / np.exp(l - l.max()).sum() if score == "softmax" else 1 / (1 + np.exp(-l))
    k, p = idx.size, s[idx]
    apart = u[:, None] - u[None, :]
    g, size = np.zeros(l.size), np.zeros(l.size)
    if renormalize:
        w = p / p.sum()
        tail = 1.0 if score == "softmax" else 1 / (1 + np.exp(l[idx]))
        g[idx] = scale * w * (apart * w).sum(1) * tail
        size[idx] = scale * w * (np.abs(apart) * w).sum(1) * tail
    elif score == "softmax":
        rest = np.delete(s, idx).sum()
        dot, most = (u * p).sum(), (np.abs(u) * p).sum()
        g, size = -scale * s * dot, scale * s * most
        g[idx] = scale * p * (u * rest + (apart * p).sum(1))
        size[idx] = scale * p * (np.abs(u) * rest + (np.abs(apart) * p).sum(1))
    else:
        g[idx] = scale * u * p / (1 + np.exp(l[idx]))
        size[idx] = np.abs(g[idx])
    return g, size


@pytest.mark.parametrize("gap", [0.0, 5.0, 10.0, 16.0, 20.0])
@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True),
                                               ("sigmoid", False)])
@pytest.mark.parametrize("T,E,k,dtype", [(20, 64, 8, torch.float32), (9, 250, 8, torch.float32),
                                         (7, 1000, 32, torch.float32), (5, 9, 2, torch.float32),
                                         (20, 128, 6, torch.bfloat16)])
def test_one_weight_dominates(cuda_device, gap, score, renormalize, T, E, k, dtype):
    gen = torch.Generator().manual_seed(E + int(gap))
    l = torch.randn((T, E), generator=gen)
    top = torch.randint(0, E, (T,), generator=gen)
    l[torch.arange(T), top] = l.max(1)[0] + gap
    if score == "sigmoid":      # scores of e^-gap beside one that is not small
        l -= gap
    x = l.to(dtype).cuda().requires_grad_(True)
    w, idx = L.route_experts(x, k, score=score, renormalize=renormalize, scale=2.5)
    u = torch.randn((T, k), generator=gen)
    g, = torch.autograd.grad(w, x, u.cuda())
    # the same through the call of the saved results
    again = L.route_backward(x.detach(), w.detach(), idx, u.cuda(), score=score, renormalize=renormalize, scale=2.5)
    assert torch.equal(g, again)
    l64, idx = x.detach().double().cpu().numpy(), idx.long().cpu().numpy()
    for t in range(T):
        want, size = expected(l64[t], idx[t], u[t].double().numpy(), score, renormalize, 2.5)
        spread = l64[t].max() - l64[t].min()
        tol = (4 * (2 * spread + 52) + 3 * (2 * k + 1) + k + 4) * 2.0 ** -24 * size + R.UNIT[dtype] * 1.01 * np.abs(want) + 1.2e-38
        off = np.abs(g[t].double().cpu().numpy() - want)
        assert (off <= tol).all(), (t, (off / np.maximum(size, 1e-300)).max())


def test_by_differences(cuda_device):
    """The dominating expert's gradient is the rate at which the loss changes: float64 central
    differences of the formula, whose own error is about h^2."""
    l = torch.tensor([[14.0, 0.5, -0.25, 1.0, 0.0, -1.0, 0.75, 0.25]], device="cuda")
    u = torch.tensor([[1.0, -0.5, 0.25, 2.0]], device="cuda")
    x = l.clone().requires_grad_(True)
    w, idx = L.route_experts(x, 4)
    g, = torch.autograd.grad(w, x, u)

    def loss(l64):
        p = np.exp(l64 - l64.max())[idx[0].cpu().numpy()]
        return (u[0].double().cpu().numpy() * (p / p.sum())).sum()

    l64 = l[0].double().cpu().numpy()
    for i in range(8):
        h = np.zeros(8)
        h[i] = 1e-3
        # the change is 1e-5 of weights near 1, each rounded to 2^-53
        slope = (loss(l64 + h) - loss(l64 - h)) / 2e-3
        assert abs(float(g[0, i]) - slope) <= 4e-6 * abs(slope) + 1e-12
