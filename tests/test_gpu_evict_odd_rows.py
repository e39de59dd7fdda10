"""Eviction of rows long enough for the sampled search whose scores are not all ordinary
numbers: NaN, infinities, zeros of both signs, denormals, heavy ties.  Positions against a
stable sort (exact), with guard words on both sides of the positions through the C call."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_selection_primitive_b200 as L

pytestmark = pytest.mark.gpu
GUARD = 4096


def order_of(x):
    """Positions by falling score, equal scores by position; NaN below every number."""
    x = x.astype(np.float64)
    return np.lexsort((np.arange(x.size), np.where(np.isnan(x), np.inf, -x), np.isnan(x)))


def scores(n, seed, shares):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(n).astype(np.float32)
    at = rng.permutation(n)
    for value, m in shares.items():
        m = int(round(m * n)) if m <= 1 else m
        here, at = at[:m], at[m:]
        if value == "tiny":
            x[here] = rng.choice([-1, 1], m) * rng.integers(0, 5, m) * np.float32(1.4e-45)
        elif value == "zeros":
            x[here] = rng.choice([-0.0, 0.0], m)
        else:
            x[here] = {"nan": np.nan, "low": -np.inf, "high": np.inf,
                       "lowest": np.finfo(np.float32).min}[value]
    return x


def run(rows, budget, first, last):
    """(positions, lengths) of the rows through lapsum_evict, the guard words looked at."""
    H, n = rows.shape
    s = torch.from_numpy(rows).cuda()
    k = torch.arange(H * n, device="cuda", dtype=torch.float32).view(1, H, n, 1)
    v = -k
    lengths = torch.tensor([n], dtype=torch.int32, device="cuda")
    room = torch.full((2 * GUARD + H * budget,), -77, dtype=torch.int32, device="cuda")
    pos = room[GUARD:GUARD + H * budget]
    ko, vo = k.new_empty((1, H, budget, 1)), k.new_empty((1, H, budget, 1))
    so, left = k.new_empty((1, H, budget)), torch.empty_like(lengths)
    strides = (ctypes.c_int64 * 16)(H * n, n, 1, H * n, n, 1, H * n, n, H * budget, budget, 1,
                                    H * budget, budget, 1, H * budget, budget)
    code = L._lib().lapsum_evict(k.data_ptr(), v.data_ptr(), 0, s.data_ptr(), lengths.data_ptr(), strides,
                                 1, H, n, 1, budget, first, last, ko.data_ptr(), vo.data_ptr(), so.data_ptr(),
                                 pos.data_ptr(), left.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert code == 0
    torch.cuda.synchronize()
    assert (room[:GUARD] == -77).all() and (room[GUARD + H * budget:] == -77).all()
    pos = pos.view(H, budget)
    at = pos.long()
    assert torch.equal(ko[0, :, :, 0], k[0, :, :, 0].gather(1, at)) and torch.equal(vo, -ko)
    bits = lambda t: t.contiguous().view(torch.int32)  # noqa: E731
    assert torch.equal(bits(so[0]), bits(s).gather(1, at))
    return pos.cpu().numpy(), int(left[0])


def check(rows, budget, first=0, last=0):
    n = rows.shape[1]
    got, left = run(rows, budget, first, last)
    assert left == budget
    for h, x in enumerate(rows):
        mid = order_of(x[first:n - last])[:budget - first - last] + first
        want = np.sort(np.concatenate([np.arange(first), mid, np.arange(n - last, n)]))
        assert np.array_equal(got[h], want), (h, budget)


SHARES = [{"nan": 0.1}, {"nan": 0.6}, {"low": 0.1}, {"low": 0.6}, {"nan": 0.3, "low": 0.3},
          {"high": 0.3, "low": 0.2, "nan": 0.2}, {"zeros": 0.6, "low": 0.015}, {"tiny": 0.9},
          {"tiny": 0.5, "nan": 0.2}, {"lowest": 0.5, "low": 0.2}, {"nan": 1.0}, {"low": 1.0},
          {"zeros": 1.0}]


@pytest.mark.parametrize("n", [2049, 4096, 20000, 70001])
@pytest.mark.parametrize("shares", SHARES)
def test_evict_odd_scores_of_long_rows(cuda_device, n, shares):
    rows = np.stack([scores(n, n + h, shares) for h in range(2)])
    x = rows[0]
    edges = {1, n // 2, n - 1, int(n * 0.99)}
    ordinary = int(np.isfinite(x).sum())
    for edge in (int((x == np.inf).sum()), ordinary, int((~np.isnan(x)).sum()), int((x > 0).sum())):
        edges |= {edge - 1, edge, edge + 1}
    for budget in sorted(e for e in edges if 1 <= e < n):
        check(rows, budget)
        if budget > 50:
            check(rows, budget, 4, 33)


@pytest.mark.parametrize("n,budget,shares", [
    (5000, 4000, {"nan": 3000}), (20000, 19800, {"low": 300, "zeros": 12000}),
    (20030, 20020, {"low": 30, "zeros": 20000}), (1000000, 997500, {"low": 5000}),
    (1000000, 997500, {"nan": 5000}), (1000000, 992000, {"nan": 5000, "low": 5000})])
def test_evict_boundary_among_odd_scores(cuda_device, n, budget, shares):
    """A boundary among -inf or NaN, more of them, or of ties above, than the list holds."""
    check(np.stack([scores(n, 3 * n + h, shares) for h in range(2)]), budget)


def test_evict_masked_scores_through_the_binding(cuda_device):
    """Keys masked with -inf go first, as a caller uses it."""
    B, H, n = 2, 3, 30000
    gen = torch.Generator().manual_seed(5)
    s = torch.rand((B, H, n), generator=gen)
    s[:, :, torch.randperm(n, generator=gen)[:9000]] = -float("inf")
    s[1, 1] = float("nan")
    k = torch.randn((B, H, n, 16), generator=gen).to(torch.bfloat16).cuda()
    e = L.evict(k, k.clone(), s.cuda(), torch.tensor([n, n], dtype=torch.int32).cuda(), 25000, first=3, last=70)
    for b in range(B):
        for h in range(H):
            mid = order_of(s[b, h, 3:n - 70].numpy())[:25000 - 73] + 3
            want = np.sort(np.concatenate([np.arange(3), mid, np.arange(n - 70, n)]))
            assert np.array_equal(e.positions[b, h].cpu().numpy(), want)
