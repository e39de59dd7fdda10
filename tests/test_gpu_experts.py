"""Expert routing and expert rows against 64-bit plain forms (tests/select_reference.py).

Tolerances, counted in roundings.  A weight is exp(l - m) (the subtraction is off
by |l - m| 2^-24, the exponential by two units) over a sum of at most 1024 terms
(32 in a lane, five levels across lanes, each term off like the numerator), times
the scale: relative error at most (2 |l - m| + 40 + 12) 2^-24.  Gradients are
products of weights, upstream values and one dot product over k.
"""
import numpy as np
import pytest
import torch

import sparse_selection_primitive_b200 as L
from tests import select_reference as R

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def check_route(logits, k, seed=0, **how):
    """Forward and backward of one call against the rows' references."""
    T, E = logits.shape
    bias = how.get("bias")
    x = logits.detach().requires_grad_(True)
    w, idx = L.route_experts(x, k, **how)
    u = torch.randn((T, k), generator=torch.Generator().manual_seed(seed)).cuda()
    g, = torch.autograd.grad(w, x, u)
    assert w.shape == idx.shape == (T, k) and w.dtype == torch.float32 and idx.dtype == torch.int32
    assert g.dtype == logits.dtype and g.shape == logits.shape
    ref = dict(how, bias=None if bias is None else bias.double().cpu().numpy())
    grad_how = (how.get("score", "softmax"), how.get("renormalize", True), how.get("scale", 1.0))
    l64, w, idx = logits.detach().double().cpu().numpy(), w.detach().cpu().double().numpy(), idx.cpu().numpy()
    g, u = g.double().cpu().numpy(), u.double().cpu().numpy()
    for t in range(T):
        w_ref, i_ref, s = R.route_row(l64[t], k, **ref)
        assert np.array_equal(idx[t], i_ref), (t, idx[t], i_ref)
        if s is None:
            assert np.isnan(w[t]).all() and np.isnan(g[t]).all()
            continue
        live = l64[t][l64[t] > -np.inf]
        spread = min(float(live.max() - live.min()), 110.0) if live.size else 0.0
        rel = (2 * spread + 52) * 2.0 ** -24
        # below the smallest normal number a result may be flushed to 0
        assert (np.abs(w[t] - w_ref) <= rel * w_ref + 1.2e-38).all(), (t, w[t], w_ref)
        g_ref = R.route_grad_row(l64[t], i_ref, u[t], *grad_how)
        size = np.abs(u[t] * w_ref).sum() + np.abs(w_ref * u[t]).max(initial=0)
        # each element: s_i or w_i times a sum over k, both off by rel and (k + 4) units
        tol = (4 * rel + (2 * k + 8) * 2.0 ** -24) * size + R.UNIT[logits.dtype] * np.abs(g_ref) * 1.01 + 6e-8 * (logits.dtype == torch.float16)
        assert (np.abs(g[t] - g_ref) <= tol + 1.2e-38).all(), (t, np.abs(g[t] - g_ref).max(), tol)


def rows(seed, T, E, dtype, scale=1.5):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn((T, E), generator=gen) * scale).to(dtype).cuda()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 2, 2), (5, 8, 3), (9, 33, 32), (70, 64, 6),
                                   (33, 100, 5), (64, 256, 8), (4, 257, 1), (3, 1000, 12),
                                   (2, 1024, 32)])
def test_route_plain(cuda_device, dtype, T, E, k):
    check_route(rows(E + k, T, E, dtype), k)
    check_route(rows(E + k + 1, T, E, dtype), k, renormalize=False, scale=0.5)
    check_route(rows(E + k + 2, T, E, dtype), k, score="sigmoid", scale=2.5)
    check_route(rows(E + k + 3, T, E, dtype), k, score="sigmoid", renormalize=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top,group_top,k", [(64, 8, 3, 2, 6), (256, 8, 4, 2, 8),
                                                      (24, 3, 1, 1, 5), (160, 5, 2, 2, 4),
                                                      (32, 32, 7, 2, 7), (1024, 32, 5, 1, 32),
                                                      (100, 2, 1, 2, 9), (96, 1, 1, 2, 4)])
def test_route_bias_and_groups(cuda_device, score, E, groups, top, group_top, k):
    gen = torch.Generator().manual_seed(E)
    bias = (torch.randn(E, generator=gen) * 0.05).cuda()
    for b in (bias, None):
        for dtype in (torch.float32, torch.bfloat16):
            check_route(rows(7 * E + k, 40, E, dtype), k, score=score, bias=b, groups=groups,
                        top_groups=top, group_top=group_top)


def test_route_ties_and_near_ties(cuda_device):
    """Equal logits go to the lower index; keys that fp32 cannot tell apart are
    ordered as their 64-bit values are."""
    check_route(torch.zeros((4, 256), device="cuda"), 8)
    check_route(torch.zeros((4, 256), device="cuda"), 8, score="sigmoid", groups=8, top_groups=4,
                bias=torch.zeros(256, device="cuda"))
    check_route(rows(3, 50, 128, torch.float32).round(), 10)
    check_route(rows(4, 50, 128, torch.float32).round(), 10, groups=4, top_groups=2)
    # logits a few ulp apart: the scores round to the same fp32 value
    base = torch.full((32, 96), 3.0) + torch.arange(96) * 2.0 ** -22
    x = base[:, torch.randperm(96, generator=torch.Generator().manual_seed(5))].cuda()
    check_route(x, 7)
    check_route(x, 7, score="sigmoid", bias=torch.zeros(96, device="cuda"))
    check_route(x, 7, score="softmax", bias=torch.full((96,), 0.25, device="cuda"), groups=8,
                top_groups=3)
    # -0 and +0 are one value
    z = torch.zeros((2, 40))
    z[:, ::2] = -0.0
    check_route(z.cuda(), 5)


@pytest.mark.parametrize("how", [dict(), dict(renormalize=False), dict(score="sigmoid"),
                                 dict(score="sigmoid", bias=True, groups=4, top_groups=2),
                                 dict(bias=True)])
def test_route_masked_rows(cuda_device, how):
    """-inf logits are never chosen; rows with too few others hold -1 and 0; rows with a
    NaN or +inf hold -1 and NaN; the type's lowest value is an ordinary logit."""
    E, k = 32, 6
    how = dict(how)
    if how.get("bias"):
        how["bias"] = torch.linspace(-0.1, 0.1, E, device="cuda")
    for dtype in DTYPES:
        x = rows(11, 12, E, dtype).clone()
        x[0] = -float("inf")
        x[1, 3:] = -float("inf")
        x[2, ::2] = -float("inf")
        x[3, 5] = float("nan")
        x[4, 6] = float("inf")
        x[5] = torch.finfo(dtype).min
        x[6, 4:] = torch.finfo(dtype).min
        x[7, 1:] = -float("inf")
        check_route(x, k, **how)


def test_route_extreme_logits(cuda_device):
    """Scores that underflow keep the ratios of renormalised weights."""
    x = rows(12, 6, 64, torch.float32) - 200.0
    check_route(x, 4, score="sigmoid")
    check_route(rows(13, 6, 64, torch.float32) * 40, 4)
    x = rows(14, 6, 64, torch.float32) + 60.0
    check_route(x, 4, score="sigmoid")


def test_route_strided_rows(cuda_device):
    for dtype in DTYPES:
        big = rows(15, 20, 300, dtype)
        check_route(big[:, 3:103], 5)          # odd offset and stride: no packs
        check_route(big[:, :256], 5, groups=8, top_groups=2)
        check_route(big.t()[:60], 5)           # a transposed view
        check_route(big[::2, :64], 5)


def test_route_gradient_of_a_single_expert_is_zero(cuda_device):
    """One renormalised weight is the scale whatever the logits: its gradient is exactly 0."""
    for how in (dict(scale=2.5), dict(score="sigmoid", scale=0.3)):
        x = rows(18, 50, 24, torch.float32).requires_grad_(True)
        w, _ = L.route_experts(x, 1, **how)
        g, = torch.autograd.grad(w, x, torch.randn((50, 1), device="cuda"))
        assert (w == torch.tensor(how["scale"], device="cuda")).all() and (g == 0).all()


def test_route_refusals(cuda_device):
    x = rows(16, 4, 64, torch.float32)
    for bad in (dict(k=0), dict(k=33), dict(k=4, groups=5, top_groups=2),
                dict(k=4, groups=8, top_groups=9), dict(k=20, groups=8, top_groups=2),
                dict(k=4, scale=0.0), dict(k=4, scale=float("inf")),
                dict(k=4, groups=8, top_groups=2, group_top=3)):
        with pytest.raises((L.LapSumError, ValueError)):
            L.route_experts(x, **bad)
    with pytest.raises(L.LapSumError):
        L.route_experts(rows(1, 2, 1025, torch.float32), 4)
    with pytest.raises(ValueError):
        L.route_experts(x, 4, score="linear")
    with pytest.raises(TypeError):
        L.route_experts(x.double(), 4)
    with pytest.raises(ValueError):
        L.route_experts(x, 4, bias=torch.zeros(63, device="cuda"))
    w, idx = L.route_experts(x[:0], 4)
    assert w.shape == idx.shape == (0, 4)


def test_route_gradient_by_differences(cuda_device):
    """The gradient against central differences of the 64-bit form."""
    x = rows(17, 3, 20, torch.float32)
    for how in (dict(), dict(renormalize=False, scale=2.0), dict(score="sigmoid"),
                dict(score="sigmoid", renormalize=False)):
        xr = x.clone().requires_grad_(True)
        w, idx = L.route_experts(xr, 4, **how)
        u = torch.linspace(-1, 2, 12, device="cuda").view(3, 4)
        g = torch.autograd.grad(w, xr, u)[0].double().cpu().numpy()
        l64, h = x.double().cpu().numpy(), 1e-5
        for t in range(3):
            for e in range(20):
                f = []
                for s in (h, -h):
                    l = l64[t].copy()
                    l[e] += s
                    f.append(R.route_row(l, 4, **how)[0] @ u[t].double().cpu().numpy())
                # differences: h^2 of a third derivative below 10, and 2^-53 / h
                assert abs((f[0] - f[1]) / (2 * h) - g[t, e]) <= 1e-6, (how, t, e)


# --- rows --------------------------------------------------------------------------------
def assignments(seed, T, k, E, drop=0.1):
    gen = torch.Generator().manual_seed(seed)
    e = torch.randint(0, E, (T, k), generator=gen)
    e[torch.rand((T, k), generator=gen) < drop] = -1
    return e.to(torch.int32)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 256), (7, 3, 5), (256, 8, 256), (257, 8, 256),
                                   (5000, 4, 37), (700, 32, 1024), (20000, 1, 2)])
def test_plan(cuda_device, T, k, E):
    for drop in (0.0, 0.2, 1.0):
        e = assignments(T + k, T, k, E, drop)
        p = L.expert_plan(e.cuda(), E)
        offsets, slots, order = R.plan(e.numpy(), E)
        assert np.array_equal(p.offsets.cpu().numpy(), offsets)
        assert np.array_equal(p.slots.cpu().numpy(), slots)
        assert np.array_equal(p.order.cpu().numpy(), order)


def test_plan_large(cuda_device):
    """Many blocks: against torch's stable sort, with all assignments to one expert too."""
    for T, k, E, one in ((130000, 8, 300, False), (400001, 2, 16, True)):
        e = assignments(T, T, k, E, 0.05)
        if one:
            e[:] = 3
        flat = torch.where(e < 0, E, e).view(-1).cuda()
        order = flat.sort(stable=True)[1]
        p = L.expert_plan(e.cuda(), E)
        assert torch.equal(p.order.long(), order)
        assert torch.equal(p.slots.view(-1)[order].long(), torch.arange(T * k, device="cuda"))
        counts = torch.bincount(flat, minlength=E + 1)[:E].cumsum(0)
        assert torch.equal(p.offsets[1:].long(), counts) and p.offsets[0] == 0


def test_plan_out_of_range_experts_are_dropped(cuda_device):
    e = torch.tensor([[0, 5], [2 ** 31 - 1, -2 ** 31], [4, 1]], dtype=torch.int32)
    p = L.expert_plan(e.cuda(), 5)
    assert p.offsets.tolist() == [0, 1, 2, 2, 2, 3]
    assert p.slots.tolist() == [[0, 3], [4, 5], [2, 1]]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 1), (5, 2, 4, 8), (33, 8, 16, 64), (100, 3, 7, 1000),
                                     (40, 6, 64, 2049), (17, 32, 40, 36), (3, 2, 2, 4100)])
def test_rows_forward_and_backward(cuda_device, dtype, T, k, E, H):
    gen = torch.Generator().manual_seed(H)
    e = assignments(T * 3 + H, T, k, E)
    offsets, slots, order = R.plan(e.numpy(), E)
    live = int(offsets[-1])
    p = L.expert_plan(e.cuda(), E)
    x = torch.randn((T, H), generator=gen).to(dtype)
    y = torch.randn((T * k, H), generator=gen).to(dtype)
    y[live:] = float("nan")          # rows that no expert wrote may hold anything
    w = torch.rand((T, k), generator=gen)
    dxs = torch.randn((T * k, H), generator=gen).to(dtype)
    dout = torch.randn((T, H), generator=gen).to(dtype)
    xc, yc, wc = (v.cuda().requires_grad_(True) for v in (x, y, w))
    xs = L.expert_gather(xc, p)
    out = L.expert_combine(yc, wc, p)
    dx, = torch.autograd.grad(xs, xc, dxs.cuda())
    dy, dw = torch.autograd.grad(out, (yc, wc), dout.cuda())
    xs_ref = torch.zeros_like(xs.cpu())
    xs_ref[:live] = x[torch.from_numpy(order[:live] // k)]
    assert torch.equal(xs.detach().cpu(), xs_ref)
    unit = R.UNIT[dtype]
    f64 = lambda v: v.detach().cpu().double().numpy()  # noqa: E731
    on = slots < live
    y64 = np.where(np.arange(T * k)[:, None] < live, np.nan_to_num(f64(y)), 0.0)
    terms = f64(w)[..., None] * on[..., None] * y64[slots]
    o_ref, o_abs = terms.sum(1), np.abs(terms).sum(1)
    # k products and sums in fp32, one rounding to the type (fp16 below 2^-14: half a step 2^-25)
    low = 2.0 ** -25 if dtype == torch.float16 else 1e-40
    tol = (k + 1) * 2.0 ** -24 * o_abs + unit * np.abs(o_ref) * 1.01 + low
    assert (np.abs(f64(out) - o_ref) <= tol).all()
    g = np.where(on[..., None], f64(dxs)[slots], 0.0)
    tol = (k + 1) * 2.0 ** -24 * np.abs(g).sum(1) + unit * np.abs(g.sum(1)) * 1.01 + low
    assert (np.abs(f64(dx) - g.sum(1)) <= tol).all()
    dy_ref = np.zeros((T * k, H))
    dy_ref[slots.reshape(-1)] = ((f64(w) * on)[..., None] * f64(dout)[:, None]).reshape(T * k, H)
    assert (np.abs(f64(dy) - dy_ref) <= (unit + 2.0 ** -24) * np.abs(dy_ref) * 1.01 + low).all()
    prod = f64(dout)[:, None] * np.where(on[..., None], y64[slots], 0.0)
    # a thread's run and eight levels of sums
    tol = (H / 256 + 32) * 2.0 ** -24 * np.abs(prod).sum(2) + 1e-40
    assert (np.abs(f64(dw) - prod.sum(2)) <= tol).all()


def test_rows_strides_and_broadcast_gradients(cuda_device):
    T, k, E, H = 12, 3, 5, 64
    p = L.expert_plan(assignments(1, T, k, E).cuda(), E)
    big = torch.randn((T, 2 * H + 1), device="cuda")
    for x in (big[:, :H], big[:, 1:H + 1], big.t()[:H].t(), big[:1, :H].expand(T, H)):
        assert torch.equal(L.expert_gather(x, p), L.expert_gather(x.contiguous(), p))
    y = torch.randn((T * k, H), device="cuda", requires_grad=True)
    w = torch.rand((T, k), device="cuda", requires_grad=True)
    out = L.expert_combine(y, w, p)
    one = torch.autograd.grad(out, (y, w), torch.ones((), device="cuda").expand(T, H),
                              retain_graph=True)
    two = torch.autograd.grad(out, (y, w), torch.ones((T, H), device="cuda"))
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    only = torch.autograd.grad(L.expert_combine(y.detach(), w, p).sum(), w)[0]
    assert torch.equal(only, two[1])


def test_second_derivatives_are_refused(cuda_device):
    """A backward pass that is itself recorded gives its gradient, but no second one."""
    x = rows(40, 4, 16, torch.float32).requires_grad_(True)
    w, _ = L.route_experts(x, 3)
    g, = torch.autograd.grad(w.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_graph_of_a_backward_pass(cuda_device):
    """Forward and backward captured together and replayed with other inputs."""
    T, E, k, H = 20, 16, 3, 40
    x, h = torch.zeros((T, E), device="cuda"), torch.zeros((T, H), device="cuda")
    x.requires_grad_(True), h.requires_grad_(True)
    dout = torch.randn((T, H), device="cuda")

    def step(x, h):
        w, i = L.route_experts(x, k, score="sigmoid")
        p = L.expert_plan(i, E)
        out = L.expert_combine(L.expert_gather(h, p) * 2, w, p)
        return (out,) + torch.autograd.grad(out, (x, h), dout)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, h)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(x, h)
    for seed in (3, 4):
        gen = torch.Generator().manual_seed(seed)
        a, b = torch.randn((T, E), generator=gen).cuda(), torch.randn((T, H), generator=gen).cuda()
        with torch.no_grad():
            x.copy_(a)
            h.copy_(b)
        graph.replay()
        want = step(a.requires_grad_(True), b.requires_grad_(True))
        assert all(torch.equal(u, v) for u, v in zip(got, want))


def test_rows_refusals(cuda_device):
    p = L.expert_plan(assignments(1, 4, 2, 3).cuda(), 3)
    x = torch.zeros((4, 8), device="cuda")
    with pytest.raises(ValueError):
        L.expert_gather(x[:3], p)
    with pytest.raises(TypeError):
        L.expert_gather(x.double(), p)
    with pytest.raises(ValueError):
        L.expert_combine(x, torch.zeros((4, 2), device="cuda"), p)
    with pytest.raises(ValueError):
        L.expert_combine(torch.zeros((8, 8), device="cuda"), torch.zeros((4, 3), device="cuda"), p)
    with pytest.raises(TypeError):
        L.expert_combine(torch.zeros((8, 8), device="cuda"), x[:, :2].double(), p)
    with pytest.raises(TypeError):
        L.expert_plan(torch.zeros((4, 2), device="cuda", dtype=torch.int64), 3)
    with pytest.raises((ValueError, L.LapSumError)):
        L.expert_plan(torch.zeros((4, 2), device="cuda", dtype=torch.int32), 1025)
    with pytest.raises(L.LapSumError):
        L.expert_gather(x, L.expert_plan(torch.zeros((4, 33), device="cuda", dtype=torch.int32), 3))
    e = L.expert_plan(torch.zeros((0, 2), device="cuda", dtype=torch.int32), 3)
    assert L.expert_gather(x[:0], e).shape == (0, 8) and e.offsets.tolist() == [0] * 4
    assert L.expert_combine(x[:0], torch.zeros((0, 2), device="cuda"), e).shape == (0, 8)


# --- together ------------------------------------------------------------------------------
def test_mixture_of_experts_layer(cuda_device):
    """route -> plan -> gather -> the experts' products -> combine, forward and gradients
    of tokens and router, against the dense layer in float64; then the same layer captured
    and replayed with other inputs."""
    T, D, E, k = 48, 32, 12, 3
    gen = torch.Generator().manual_seed(3)
    wr = (torch.randn((D, E), generator=gen) * 0.5).cuda()
    we = (torch.randn((E, D, D), generator=gen) * 0.2).cuda()
    bias = (torch.randn(E, generator=gen) * 0.02).cuda()

    def layer(x, r):
        w, idx = L.route_experts(x @ r, k, score="sigmoid", bias=bias, groups=4, top_groups=2)
        plan = L.expert_plan(idx, E)
        xs = L.expert_gather(x, plan)
        # every row times its expert's matrix, chosen by the plan's offsets
        which = torch.bucketize(torch.arange(T * k, device="cuda", dtype=torch.int32),
                                plan.offsets[1:], right=True).clamp(max=E - 1)
        y = torch.bmm(xs[:, None, :], we[which])[:, 0]
        return L.expert_combine(y, w, plan), idx

    x = torch.randn((T, D), generator=gen).cuda().requires_grad_(True)
    r = wr.clone().requires_grad_(True)
    out, idx = layer(x, r)
    dout = torch.randn((T, D), generator=gen).cuda()
    gx, gr = torch.autograd.grad(out, (x, r), dout)
    x64, r64 = x.detach().double().requires_grad_(True), r.detach().double().requires_grad_(True)
    s = torch.sigmoid(x64 @ r64).gather(1, idx.long())
    ref = ((s / s.sum(1, keepdim=True))[..., None] *
           torch.einsum("td,tkde->tke", x64, we.double()[idx.long()])).sum(1)
    hx, hr = torch.autograd.grad(ref, (x64, r64), dout.double())
    # fp32 products over D = 32 (router, experts) and k = 3: some 80 roundings of sums of
    # terms that are up to some 8 times the result
    for a, b in ((out, ref), (gx, hx), (gr, hr)):
        assert (a.detach().double() - b.detach()).abs().max() <= 640 * 2.0 ** -24 * b.abs().max()

    xg = torch.randn((T, D), generator=gen).cuda()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream), torch.no_grad():
        layer(xg, wr)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.no_grad(), torch.cuda.graph(graph):
        got, chosen = layer(xg, wr)
    for seed in (8, 9):
        fresh = torch.randn((T, D), generator=torch.Generator().manual_seed(seed)).cuda()
        xg.copy_(fresh)
        graph.replay()
        with torch.no_grad():
            want, want_idx = layer(fresh, wr)
        assert torch.equal(got, want) and torch.equal(chosen, want_idx)


def test_soft_router_list_feeds_the_plan(cuda_device):
    """The soft top-k router's support list (unused places preset to -1) is a plan's input."""
    B, n, cap = 40, 64, 12
    r = rows(5, B, n, torch.float32)
    out = (torch.empty((B, n), device="cuda"), torch.empty(B, dtype=torch.float64, device="cuda"),
           torch.full((B, cap), -1, dtype=torch.int32, device="cuda"),
           torch.zeros((B, cap), device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda"))
    p, _, idx, vals, cnt = L.forward_router(r, 4.0, 0.05, eps=1e-3, cap=cap, out=out)
    plan = L.expert_plan(idx, n)
    assert int(plan.offsets[-1]) == int(cnt.clamp(max=cap).sum())
    x = torch.randn((B, 24), device="cuda")
    y = L.expert_combine(L.expert_gather(x, plan), vals, plan)
    # each row comes back times the sum of its listed p: cap products and sums
    want = x.double() * vals.double().sum(1, keepdim=True)
    assert ((y.double() - want).abs() <= 2 * (cap + 1) * 2.0 ** -24 * want.abs() + 1e-30).all()


def test_other_stream_and_two_calls_at_once(cuda_device):
    T, E, k, H = 300, 64, 4, 256
    x = rows(21, T, E, torch.float32)
    h = torch.randn((T, H), device="cuda")
    w0, i0 = L.route_experts(x, k)
    p0 = L.expert_plan(i0, E)
    o0 = L.expert_combine(L.expert_gather(h, p0), w0, p0)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            for _ in range(5):
                w, i = L.route_experts(x, k)
                p = L.expert_plan(i, E)
                o = L.expert_combine(L.expert_gather(h, p), w, p)
            got.append((w, i, p.order, o))
    torch.cuda.synchronize()
    for w, i, order, o in got:
        assert torch.equal(w, w0) and torch.equal(i, i0)
        assert torch.equal(order, p0.order) and torch.equal(o, o0)
