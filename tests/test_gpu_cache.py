"""Cache attention with accumulated weight, and eviction, against 64-bit plain forms.

Tolerances, counted in roundings.  A logit is a sum of D products of 16-bit values,
exact in fp32 and added in fp32: off by at most D 2^-24 of the sum of their
magnitudes, times the scale, and the softmax's exponent by that and a rounding of
its own argument; a weight's relative error is the sum of those (plus the sum of N
weights, all of one sign).  The output takes weights that may be held as pairs of
16-bit values (2^-16 relative), sums them in fp32 and is rounded once to its type.
"""
import numpy as np
import pytest
import torch

import sparse_selection_primitive_b200 as L
from tests import select_reference as R

pytestmark = pytest.mark.gpu
HALF = [torch.bfloat16, torch.float16]


def caches(seed, B, Sq, Hq, Hkv, N, D, dtype, layout="bhnd"):
    gen = torch.Generator().manual_seed(seed)
    q = (torch.randn((B, Sq, Hq, D), generator=gen) * 1.5).to(dtype)
    if layout == "bhnd":
        k, v = (torch.randn((B, Hkv, N, D), generator=gen).to(dtype) for _ in range(2))
    else:  # rows of all heads next to each other
        k, v = (torch.randn((B, N, Hkv, D), generator=gen).to(dtype).transpose(1, 2)
                for _ in range(2))
    score = torch.rand((B, Hkv, N), generator=gen)
    return q, k, v, score


def check_attend(q, k, v, lengths, score, scale=None):
    """One call against the reference; rows of the caches behind the lengths are NaN, and
    scores there have to stay."""
    B, Sq, Hq, D = q.shape
    N = k.shape[2]
    n = torch.tensor(lengths, dtype=torch.int32)
    inside = torch.arange(N)[None, None, :] < n[:, None, None]
    k, v = (torch.where(inside[..., None], c, torch.full((), float("nan"), dtype=c.dtype))
            for c in (k, v))
    # the view keeps its layout
    kc, vc = (torch.empty_strided(c.shape, o.stride(), dtype=c.dtype, device="cuda").copy_(c)
              for c, o in ((k, k), (v, v)))
    sc = score.cuda()
    args = {} if scale is None else dict(scale=scale)
    out = L.attend_accumulate(q.cuda(), kc, vc, n.cuda(), sc, **args)
    scale = D ** -0.5 if scale is None else scale
    q64, k64, v64 = (c.double().numpy() for c in (q, k, v))
    o_ref, s_ref = R.attend(q64, np.nan_to_num(k64), np.nan_to_num(v64), lengths, score.numpy(), scale)
    out, got = out.cpu().double().numpy(), sc.cpu().double().numpy()
    assert np.array_equal(got[~inside.expand_as(score).numpy()],
                          score.double().numpy()[~inside.expand_as(score).numpy()])
    reach = np.abs(q64).max() * np.abs(np.nan_to_num(k64)).max() * D * abs(scale)
    # the exponent's error is of sums of D terms whose magnitudes average to a tenth of reach
    rel = (D * reach / 10 + 2 * reach + 64) * 2.0 ** -24
    grown = s_ref - score.double().numpy()
    # relative errors hold for normal fp32 numbers only: each of a key's Sq * G weights below
    # 2^-126 (a reference of 1e-57 among them) may read as 0
    low = Sq * (Hq // k.shape[1]) * 2.0 ** -126
    off = np.abs(got - s_ref) - (rel * grown + 2.0 ** -23 * s_ref + low)
    assert (off <= 0).all(), off.max()
    unit = R.UNIT[q.dtype]
    vmax = np.abs(np.nan_to_num(v64)).max()
    tol = (rel + 2.0 ** -16) * vmax + unit * np.abs(o_ref) * 1.01 + 2.0 ** -24
    off = np.abs(out - o_ref) - tol
    assert (off <= 0).all(), off.max()
    return out, got


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("B,Sq,Hq,Hkv,N,D", [
    (1, 1, 1, 1, 1, 16), (1, 1, 4, 4, 7, 64), (2, 1, 8, 2, 129, 128), (1, 1, 8, 1, 1000, 128),
    (3, 1, 6, 2, 333, 96), (1, 1, 16, 1, 513, 256), (2, 1, 5, 1, 128, 80), (1, 1, 2, 2, 4097, 64),
    (1, 1, 40, 2, 700, 128), (1, 1, 12, 4, 255, 48), (2, 1, 64, 1, 400, 64), (1, 1, 1, 1, 383, 192)])
def test_attend_one_token(cuda_device, dtype, B, Sq, Hq, Hkv, N, D):
    q, k, v, score = caches(N + D, B, Sq, Hq, Hkv, N, D, dtype)
    check_attend(q, k, v, [N] * B, score)
    check_attend(q, k, v, [max(0, N - 3 * b - 1) for b in range(B)], score)


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("B,Sq,Hq,Hkv,N,D", [
    (1, 2, 4, 2, 10, 64), (2, 5, 6, 2, 200, 128), (1, 17, 8, 2, 300, 64), (2, 32, 4, 1, 140, 128),
    (1, 64, 2, 1, 64, 96), (1, 130, 2, 2, 131, 64), (1, 9, 24, 2, 650, 128), (2, 7, 3, 3, 5, 32)])
def test_attend_several_tokens(cuda_device, dtype, B, Sq, Hq, Hkv, N, D):
    q, k, v, score = caches(N + Sq, B, Sq, Hq, Hkv, N, D, dtype)
    check_attend(q, k, v, [N] * B, score)
    check_attend(q, k, v, [max(0, N - 60 * (b + 1)) for b in range(B)], score)


@pytest.mark.parametrize("Sq,Hq,Hkv,N,D", [(1, 8, 2, 30000, 128), (20, 4, 2, 24000, 64), (33, 8, 1, 9000, 128),
                                           (5, 12, 1, 7000, 256), (3, 2, 2, 40000, 16)])
def test_attend_long_runs(cuda_device, Sq, Hq, Hkv, N, D):
    """Many key tiles to a block: every ring and buffer comes round several times.  Against
    float64 on the device, at the tolerances of check_attend; a peak in the middle raises the
    references late."""
    B = 2
    q, k, v, score = caches(N, B, Sq, Hq, Hkv, N, D, torch.bfloat16)
    k[:, :, N // 2] = (q[:, 0, 0] * 3).to(k.dtype)[:, None]
    q, k, v, score = (x.cuda() for x in (q, k, v, score))
    n = torch.tensor([N, N - 333], dtype=torch.int32, device="cuda")
    s = score.clone()
    out = L.attend_accumulate(q, k, v, n, s)
    G = Hq // Hkv
    for b in range(B):
        m = int(n[b])
        see = torch.arange(m, device="cuda") <= (m - Sq + torch.arange(Sq, device="cuda"))[:, None]
        for h in range(Hkv):
            x = torch.einsum("igd,nd->gin", q[b].double()[:, h * G:(h + 1) * G], k[b, h, :m].double()) * D ** -0.5
            p = torch.softmax(x.masked_fill(~see, -float("inf")), 2)
            want = s.new_zeros(m, dtype=torch.float64) + score[b, h, :m].double() + p.sum((0, 1))
            reach = float(q.abs().max() * k.abs().max()) * D ** 0.5
            rel = (D * reach / 10 + 2 * reach + 64) * 2.0 ** -24
            off = (s[b, h, :m].double() - want).abs() - rel * p.sum((0, 1)) - 2.0 ** -23 * want
            assert off.max() <= Sq * G * 2.0 ** -126
            o = torch.einsum("gin,nd->igd", p, v[b, h, :m].double())
            tol = (rel + 2.0 ** -16) * float(v.abs().max()) + R.UNIT[q.dtype] * 1.01 * o.abs() + 2.0 ** -24
            assert ((out[b, :, h * G:(h + 1) * G].double() - o).abs() <= tol).all()
        assert torch.equal(s[b, :, m:], score[b, :, m:])


def test_attend_empty_and_short_sequences(cuda_device):
    """Lengths of zero and one, shorter than Sq, beyond N and below 0."""
    q, k, v, score = caches(1, 6, 3, 4, 2, 150, 64, torch.bfloat16)
    out, got = check_attend(q, k, v, [0, 1, 2, 3, 150, 130], score)
    assert (out[0] == 0).all() and (out[1, :2] == 0).all()
    n = torch.tensor([1000, -5, 3, 3, 3, 3], dtype=torch.int32).cuda()
    s1, s2 = score.cuda(), score.cuda()
    a = L.attend_accumulate(q.cuda(), k.cuda(), v.cuda(), n, s1)
    b = L.attend_accumulate(q.cuda(), k.cuda(), v.cuda(), n.clamp(0, 150), s2)
    assert torch.equal(a, b) and torch.equal(s1, s2)


def test_attend_views_and_layouts(cuda_device):
    q, k, v, score = caches(2, 2, 2, 8, 2, 210, 128, torch.bfloat16, layout="bnhd")
    check_attend(q, k, v, [210, 77], score)
    # a cache with room behind, heads sliced out of a wider projection, a score view
    wide = torch.randn((2, 2, 12, 128)).to(torch.bfloat16).cuda()
    cache = torch.randn((2, 2, 2, 512, 128)).to(torch.bfloat16).cuda()
    big = torch.rand((2, 2, 1024), device="cuda")
    n = torch.tensor([300, 512], dtype=torch.int32, device="cuda")
    s1, s2 = big[:, :, 100:612], big[:, :, 100:612].contiguous()
    keep = big.clone()
    a = L.attend_accumulate(wide[:, :, 2:10], cache[0], cache[1], n, s1)
    b = L.attend_accumulate(wide[:, :, 2:10].contiguous(), cache[0].clone(), cache[1].clone(), n, s2)
    assert torch.equal(a, b) and torch.equal(s1, s2)
    assert torch.equal(big[:, :, :100], keep[:, :, :100]) and torch.equal(big[:, :, 612:], keep[:, :, 612:])
    # one key/value head broadcast over the heads' dimension
    c, d = L.attend_accumulate(wide[:, :, :4], cache[0][:, :1].expand(2, 2, 512, 128),
                               cache[1][:, :1].expand(2, 2, 512, 128), n, s2.clone()), None
    d = L.attend_accumulate(wide[:, :, :4], cache[0][:, :1].repeat(1, 2, 1, 1),
                            cache[1][:, :1].repeat(1, 2, 1, 1), n, s2.clone())
    assert torch.equal(c, d)


def test_attend_score_out_and_scale(cuda_device):
    q, k, v, score = caches(3, 2, 1, 4, 2, 300, 64, torch.float16)
    check_attend(q, k, v, [300, 9], score, scale=0.3)
    check_attend(q, k, v, [300, 9], score, scale=0.0)
    n = torch.tensor([300, 9], dtype=torch.int32).cuda()
    s = score.cuda()
    into = torch.full_like(s, 7.0)
    a = L.attend_accumulate(q.cuda(), k.cuda(), v.cuda(), n, s, score_out=into)
    assert torch.equal(s, score.cuda()) and (into[1, :, 9:] == 7.0).all()
    out = torch.empty_like(a)
    b = L.attend_accumulate(q.cuda(), k.cuda(), v.cuda(), n, s, out=out)
    assert b is out and torch.equal(a, b) and torch.equal(s[0], into[0])


def test_attend_single_dimensions_with_odd_strides(cuda_device):
    """The stride of a dimension of one element means nothing."""
    n = torch.tensor([90], dtype=torch.int32, device="cuda")
    q, k, v, score = (x.cuda() for x in caches(8, 1, 1, 2, 1, 90, 64, torch.bfloat16))
    odd = lambda x, s: x.as_strided(x.shape, s)  # noqa: E731
    a = L.attend_accumulate(q, k, v, n, s1 := score.clone())
    b = L.attend_accumulate(odd(q, (3, 7, 64, 1)), odd(k, (5, 9, 64, 1)), odd(v, (1, 1, 64, 1)), n,
                            odd(s2 := score.clone(), (3, 3, 1)))
    assert torch.equal(a, b) and torch.equal(s1, s2)
    e = L.evict(k, v, score, n, 20)
    f = L.evict(odd(k, (5, 9, 64, 1)), odd(v, (1, 1, 64, 1)), odd(score, (3, 3, 1)), n, 20)
    assert all(torch.equal(x, y) for x, y in zip(e, f))


def test_cache_calls_do_not_cut_graphs(cuda_device):
    q, k, v, score = (x.cuda() for x in caches(9, 1, 1, 2, 1, 40, 64, torch.bfloat16))
    n = torch.tensor([40], dtype=torch.int32, device="cuda")
    q.requires_grad_(True)
    with pytest.raises(RuntimeError):
        L.attend_accumulate(q, k, v, n, score)
    with torch.no_grad():
        L.attend_accumulate(q, k, v, n, score)
    k.requires_grad_(True)
    with pytest.raises(RuntimeError):
        L.evict(k, v, score, n, 4)
    L.evict(k.detach(), v, score, n, 4)


def test_cache_calls_on_empty_batches(cuda_device):
    q, k, v, score = (x.cuda() for x in caches(10, 2, 1, 2, 1, 40, 64, torch.bfloat16))
    n = torch.tensor([40, 40], dtype=torch.int32, device="cuda")
    assert L.attend_accumulate(q[:0], k[:0], v[:0], n[:0], score[:0]).shape == (0, 1, 2, 64)
    out = L.attend_accumulate(q, k[:, :, :0], v[:, :, :0], n, score[:, :, :0])
    assert (out == 0).all()
    with pytest.raises(ValueError):
        L.attend_accumulate(q[:, :0], k, v, n, score)
    e = L.evict(k[:0], v[:0], score[:0], n[:0], 4)
    assert e.k.shape == (0, 1, 4, 64) and e.lengths.shape == (0,)


def test_attend_sharp_and_flat_rows(cuda_device):
    """Logits hundreds apart (weights that underflow), equal keys, and one hot key in the last place."""
    q, k, v, score = caches(4, 1, 1, 4, 1, 600, 64, torch.bfloat16)
    score.zero_()
    out, got = check_attend(q * 8, k * 4, v, [600], score)
    same = k[:, :, :1].expand_as(k).contiguous()
    out, got = check_attend(q, same, v, [600], score)
    hot = k * 0.01
    hot[0, 0, 599] = (q[0, 0, 0] * 40).to(hot.dtype)
    check_attend(q, hot, v, [600], score)


def test_attend_refusals(cuda_device):
    q, k, v, score = (c.cuda() for c in caches(5, 2, 1, 4, 2, 40, 64, torch.bfloat16))
    n = torch.tensor([40, 40], dtype=torch.int32).cuda()
    ok = lambda **o: L.attend_accumulate(**{**dict(q=q, k=k, v=v, lengths=n, score=score), **o})  # noqa: E731
    ok()
    for bad in (dict(q=q.float()), dict(q=q.half()), dict(k=k.float()), dict(lengths=n.long()),
                dict(score=score.double()), dict(q=q.cpu())):
        with pytest.raises(TypeError):
            ok(**bad)
    for bad in (dict(q=q[:, :, :3]), dict(v=v[:, :, :39]), dict(score=score[:, :, :39]),
                dict(lengths=n[:1]), dict(k=k[..., :32]), dict(q=q[:1]),
                dict(score_out=score[:, :, :1].expand_as(score)), dict(out=q),
                dict(score=score[:1].expand(2, 2, 40)), dict(out=torch.empty_like(q)[:1])):
        with pytest.raises(ValueError):
            ok(**bad)
    with pytest.raises(ValueError):   # half an overlap
        big = torch.zeros((2, 2, 50), device="cuda")
        ok(score=big[:, :, :40], score_out=big[:, :, 5:45])
    for D in (8, 24, 272):            # no multiple of 16, or too wide
        w = torch.zeros((1, 1, 4, D), dtype=torch.bfloat16, device="cuda")
        with pytest.raises(L.LapSumError):
            L.attend_accumulate(w[:, :, :1], w, w, n[:1], torch.zeros((1, 1, 4), device="cuda"))
    off = torch.zeros(2 * 2 * 40 * 64 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(2, 2, 40, 64)
    with pytest.raises(L.LapSumError):  # rows that do not start on 16 bytes
        ok(k=off)


def check_evict(k, v, score, lengths, budget, first=0, last=0, out=None):
    B, H, N, D = k.shape
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    e = L.evict(k, v, score, n, budget, first=first, last=last, out=out)
    pos = e.positions.cpu().numpy()
    s = score.cpu().numpy()
    for b in range(B):
        m = min(max(int(lengths[b]), 0), N)
        assert int(e.lengths[b]) == min(m, budget)
        for h in range(H):
            ref = R.evict_positions(s[b, h, :m], m, budget, first, last)
            assert np.array_equal(pos[b, h, :ref.size], ref), (b, h)
            assert (pos[b, h, ref.size:] == -1).all()
            at = torch.from_numpy(ref).to(k.device)
            bits = lambda t: t.contiguous().view(torch.int32 if t.element_size() == 4 else torch.int16)  # noqa: E731
            if ref.size:
                assert torch.equal(bits(e.k[b, h, :ref.size]), bits(k[b, h, at]))
                assert torch.equal(bits(e.v[b, h, :ref.size]), bits(v[b, h, at]))
                assert torch.equal(bits(e.score[b, h, :ref.size]), bits(score[b, h, at]))
            for x in (e.k, e.v, e.score):
                assert (x[b, h, ref.size:budget] == 0).all()
    return e


def evict_inputs(seed, B, H, N, D, dtype, kind="normal"):
    gen = torch.Generator().manual_seed(seed)
    k, v = (torch.randn((B, H, N, D), generator=gen).to(dtype).cuda() for _ in range(2))
    s = torch.randn((B, H, N), generator=gen)
    if kind == "ties":
        s = (s * 4).round() / 4
    if kind == "small":
        s = (s * 3 - 12).exp()
    if kind == "same":
        s = torch.ones_like(s)
    return k, v, s.cuda()


@pytest.mark.parametrize("kind", ["normal", "ties", "small", "same"])
@pytest.mark.parametrize("B,H,N,D,budget,first,last", [
    (1, 1, 1, 1, 1, 0, 0), (1, 2, 10, 8, 3, 1, 1), (2, 2, 513, 64, 100, 4, 16), (1, 3, 700, 96, 512, 0, 0),
    (2, 1, 5000, 16, 1024, 4, 128), (1, 1, 20000, 4, 1, 0, 0), (1, 1, 20000, 4, 19999, 0, 1),
    (1, 2, 1025, 128, 1025, 3, 7), (1, 1, 9000, 24, 40, 8, 32)])
def test_evict(cuda_device, kind, B, H, N, D, budget, first, last):
    for dtype in (torch.bfloat16, torch.float32):
        k, v, s = evict_inputs(N + D, B, H, N, D, dtype, kind)
        check_evict(k, v, s, [max(1, N - 37 * b) for b in range(B)], budget, first, last)


@pytest.mark.parametrize("n,budget,kind", [
    (9000, 4000, "normal"), (70001, 1024, "normal"), (70001, 35000, "normal"), (70001, 69990, "small"),
    (70001, 3, "ties"), (70001, 30000, "same"), (70001, 20000, "ties"), (300000, 70000, "normal"),
    (300000, 500, "ties"), (600001, 300000, "small"), (600001, 20, "same"), (70001, 9, "hidden"),
    (300000, 9, "hidden")])
def test_evict_long_rows(cuda_device, n, budget, kind):
    """Rows beyond the list and beyond one window of the bit maps, with samples that
    bracket, that miss (a few large scores among equal ones) and that hold too many ties:
    positions against numpy's stable sort."""
    gen = torch.Generator().manual_seed(n + budget)
    s = torch.randn((1, 2, n + 3), generator=gen)
    if kind == "ties":
        s = (s * 2).round() / 2
    if kind == "small":
        s = (s * 5 - 20).exp()
    if kind == "same":
        s = torch.ones_like(s)
    if kind == "hidden":
        s = torch.full_like(s, 0.25)
        s[0, 0, 5000:5006] = 2.0
        s[0, 1, -40:-20] = torch.arange(20) + 1.0
    s = s.cuda()[:, :, 3:]      # rows off a 16-byte boundary
    first, last = (2, 5) if budget > 8 else (0, 0)
    k = torch.randn((1, 2, n, 8), generator=gen).to(torch.bfloat16).cuda()
    e = L.evict(k, k.clone(), s, torch.tensor([n], dtype=torch.int32).cuda(), budget, first=first, last=last)
    for h in range(2):
        x = s[0, h].cpu().numpy().astype(np.float64)
        x[:first] = np.inf
        x[n - last:] = np.inf
        want = np.sort(np.argsort(-x, kind="stable")[:budget])
        assert np.array_equal(e.positions[0, h].cpu().numpy(), want)
        at = torch.from_numpy(want).cuda()
        assert torch.equal(e.k[0, h], k[0, h, at]) and torch.equal(e.score[0, h], s[0, h, at])


def test_caches_beyond_32_bit_offsets(cuda_device):
    """A cache of more than 2^31 elements a head: one key near its end takes nearly all of the
    weight, and the keys that stay lie near both ends."""
    N, D = (1 << 24) + 4321, 128 + 16
    assert N * D > 2 ** 31
    k = torch.zeros((1, 1, N, D), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    v[0, 0, -4000:].normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    n = torch.tensor([N - 7], dtype=torch.int32, device="cuda")
    hot = N - 1234
    for Hq in (2, 20):      # both kernels: few and many rows a key
        q = torch.full((1, 1, Hq, D), 1.0, dtype=torch.bfloat16, device="cuda")
        k[0, 0, hot] = 5.0  # a logit of 5 sqrt(D) = 60 against 0: the others' weights sum to 2^24 e^-60
        score = torch.zeros((1, 1, N), device="cuda")
        out = L.attend_accumulate(q, k, v, n, score)
        assert (out[0, 0] == v[0, 0, hot]).all()
        # one weight of 1 (the others below 1e-18), off by the 20 roundings of its sum and Hq sums,
        # and by those of its exponent: the logit is 60 log2(e) = 87 in powers of two, which the
        # scaling, the row's log of the sum and their difference each round to 87 2^-24, times ln 2
        assert abs(float(score[0, 0, hot]) - Hq) <= Hq * (Hq + 20 + 3 * 87 * 0.7) * 2.0 ** -24
        assert float(score[0, 0, N - 7:].abs().max()) == 0
        assert float(score[0, 0, :hot].max()) <= 1e-18
    score = torch.zeros((1, 1, N), device="cuda")
    want = [0, 1, 77, 1 << 22, N - 4000, hot, N - 9, N - 8]
    score[0, 0, want[2:6]] = torch.tensor([1.0, 2.0, 3.0, 1.0], device="cuda")
    e = L.evict(k, v, score, n, 8, first=2, last=2)
    assert e.positions[0, 0].tolist() == want
    at = torch.tensor(want, device="cuda")
    assert torch.equal(e.k[0, 0], k[0, 0, at]) and torch.equal(e.v[0, 0], v[0, 0, at])


def test_evict_short_rows(cuda_device):
    """Lengths of zero, one, the budget and one more; lengths beyond N and below 0."""
    k, v, s = evict_inputs(1, 7, 2, 64, 32, torch.float16)
    check_evict(k, v, s, [0, 1, 10, 11, 64, 99, -3], 10, 2, 3)
    check_evict(k, v, s, [0, 1, 10, 11, 64, 99, -3], 100, 2, 3)  # a budget above N


def test_evict_odd_scores(cuda_device):
    """NaN below every number, infinities, -0 equal to +0, denormals."""
    k, v, s = evict_inputs(2, 1, 4, 300, 8, torch.bfloat16)
    s[0, 0, ::3] = float("nan")
    s[0, 1, ::2] = float("inf")
    s[0, 1, 1::4] = -float("inf")
    s[0, 2] = torch.where(torch.arange(300, device="cuda") % 2 == 0, 0.0, -0.0)
    s[0, 3] = torch.arange(300, device="cuda") * 1e-44
    for budget in (1, 50, 199, 260, 299):
        check_evict(k, v, s, [300], budget, 0, 0)
    s[:] = float("nan")
    check_evict(k, v, s, [300], 7, 1, 1)


def test_evict_views_and_out(cuda_device):
    B, H, N, D, budget = 2, 3, 400, 40, 64
    base = torch.randn((2, B, N, H, D)).to(torch.bfloat16).cuda()
    k, v = base[0].transpose(1, 2), base[1].transpose(1, 2)
    score = torch.randn((B, N, H), device="cuda").transpose(1, 2)
    with pytest.raises(ValueError):      # scores of a head must be consecutive
        L.evict(k, v, score, torch.tensor([N] * B, dtype=torch.int32).cuda(), budget)
    score = torch.randn((B, H, N + 9), device="cuda")[:, :, 5:N + 5]
    check_evict(k, v, score, [N, 200], budget, 2, 8)
    room = torch.full((2, B, budget + 50, H, D), 3.0, dtype=torch.bfloat16, device="cuda")
    so = torch.full((B, H, budget + 50), 3.0, device="cuda")
    out = (room[0].transpose(1, 2), room[1].transpose(1, 2), so)
    e = check_evict(k, v, score, [N, 20], budget, 2, 8, out=out)
    assert e.k is out[0] and (e.k[:, :, budget:] == 3).all() and (e.v[:, :, budget:] == 3).all()
    assert (so[:, :, budget:] == 3).all()
    odd = torch.randn((B, H, N, 41), device="cuda")[..., 1:]      # rows off 8 and 16 bytes
    check_evict(odd, odd.clone(), score, [N, 20], budget)


def test_evict_refusals(cuda_device):
    k, v, s = evict_inputs(3, 1, 2, 40, 16, torch.bfloat16)
    n = torch.tensor([40], dtype=torch.int32).cuda()
    for bad in (dict(budget=0), dict(budget=5, first=3, last=3), dict(budget=5, first=-1)):
        with pytest.raises(ValueError):
            L.evict(k, v, s, n, **bad)
    with pytest.raises(ValueError):
        L.evict(k, v, s, n, 8, out=(k, v, s))
    with pytest.raises(ValueError):
        L.evict(k, v[:, :, :39], s, n, 8)
    with pytest.raises(TypeError):
        L.evict(k, v.float(), s, n, 8)
    with pytest.raises(ValueError):      # room for fewer rows than the budget
        L.evict(k, v, s, n, 8, out=(torch.empty_like(k)[:, :, :7], torch.empty_like(v), torch.empty_like(s)))


def test_decode_with_eviction(cuda_device):
    """A run of decoding steps over a cache: append a key, attend and accumulate, evict when
    the cache is full, go on over the compacted cache -- against the same run in float64."""
    B, H, G, D, C, budget, steps = 2, 2, 3, 64, 96, 40, 90
    gen = torch.Generator().manual_seed(9)
    kc, vc = (torch.full((B, H, C, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    spare = (torch.full_like(kc, float("nan")), torch.full_like(vc, float("nan")),
             torch.zeros((B, H, C), device="cuda"))
    sc = torch.zeros((B, H, C), device="cuda")
    n = 0
    for step in range(steps):
        q = (torch.randn((B, 1, H * G, D), generator=gen) * 1.5).to(torch.bfloat16).cuda()
        kc[:, :, n], vc[:, :, n] = (torch.randn((B, H, D), generator=gen).to(torch.bfloat16).cuda() for _ in range(2))
        sc[:, :, n] = 0
        n += 1
        lengths = torch.full((B,), n, dtype=torch.int32, device="cuda")
        before = sc.clone()
        out = L.attend_accumulate(q, kc, vc, lengths, sc)
        o_ref, s_ref = R.attend(q.double().cpu().numpy(), kc.double().nan_to_num().cpu().numpy(),
                                vc.double().nan_to_num().cpu().numpy(), [n] * B,
                                before.cpu().numpy(), D ** -0.5)
        # logits of 64 products: errors of the weights below 2^-12; out rounded to bf16
        assert np.abs(out.double().cpu().numpy() - o_ref).max() <= 4.5 * (2.0 ** -8 + 2.0 ** -12)
        assert np.abs(sc.double().cpu().numpy() - s_ref).max() <= 2.0 ** -12 * G
        if n == C:
            e = check_evict(kc, vc, sc, [n] * B, budget, 2, 8, out=spare)
            spare, (kc, vc, sc) = (kc, vc, sc), (e.k, e.v, e.score)
            n = budget
    assert n < C


def test_cache_other_streams_and_capture(cuda_device):
    q, k, v, score = (c.cuda() for c in caches(6, 2, 2, 8, 2, 500, 64, torch.bfloat16))
    n = torch.tensor([500, 123], dtype=torch.int32).cuda()

    def step(s):
        o = L.attend_accumulate(q, k, v, n, s)
        return (o, s) + tuple(L.evict(k, v, s, n, 64, first=2, last=10))

    want = step(score.clone())
    torch.cuda.synchronize()
    got = []
    for stream in (torch.cuda.Stream(), torch.cuda.Stream()):
        with torch.cuda.stream(stream):
            for _ in range(4):
                r = step(score.clone())
            got.append(r)
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))
    # two graphs over the same inputs, replayed in turn with other contents
    graphs = []
    for _ in range(2):
        s = score.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            r = step(s)
        graphs.append((g, s, r))
    for seed in (1, 2):
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(seed)))
        n.copy_(torch.tensor([400 + seed, 10 * seed], dtype=torch.int32))
        want = step(score.clone())
        for g, s, r in graphs:
            s.copy_(score)
            g.replay()
            assert all(torch.equal(a, b) for a, b in zip(r, want))


def test_attend_is_repeatable(cuda_device):
    """No result depends on the order in which blocks run."""
    q, k, v, score = (c.cuda() for c in caches(7, 2, 3, 8, 2, 3000, 128, torch.bfloat16))
    n = torch.tensor([3000, 1777], dtype=torch.int32).cuda()
    first = None
    for _ in range(5):
        s = score.clone()
        o = L.attend_accumulate(q, k, v, n, s)
        if first is None:
            first = (o, s)
        assert torch.equal(o, first[0]) and torch.equal(s, first[1])
