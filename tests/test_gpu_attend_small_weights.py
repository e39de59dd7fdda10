"""Cache attention where small weights matter: a key that takes nearly all of the weight and
whose value is 0 beside many keys of little weight, runs of many tiles in fp16, and logits
that rise from tile to tile.  Against float64 on the device.

Tolerances.  A logit is a sum of D products, off by D 2^-24 of their magnitudes' sum, and the
scaling, the reference and the exponential's own argument each round |x| log2(e) once (ln 2
each in e^x): a weight's relative error is about (D + 3) |x| 2^-24 plus 64 units for the sums.
Weights are pairs of 16-bit values: off by 2^-15 of themselves (bf16), or by 2^-22 of
themselves and 2^-48 of the row's largest (fp16; 2^-36 past 16 rows a key with D > 128).  The matrix
unit adds 16 products at a time to an fp32 sum, each addition off by a unit of 2^-23 at most.
The output is rounded once."""
import pytest
import torch

import sparse_selection_primitive_b200 as L
from tests import select_reference as R

pytestmark = pytest.mark.gpu
HALF = [torch.bfloat16, torch.float16]


def reference(q, k, v, n, score, scale):
    """(out, score, sum of p |v|) in float64, one sequence and head: q (Sq, G, D)."""
    Sq, D = q.shape[0], q.shape[2]
    k, v = k[:n].double(), v[:n].double()
    see = torch.arange(n, device=q.device) <= (n - Sq + torch.arange(Sq, device=q.device))[:, None]
    out, size = (torch.zeros(q.shape, dtype=torch.float64, device=q.device) for _ in range(2))
    grown = torch.zeros(n, dtype=torch.float64, device=q.device)
    for g in range(q.shape[1]):
        x = (q[:, g].double() @ k.t()) * scale
        p = torch.softmax(x.masked_fill(~see, -float("inf")), 1)
        out[:, g], size[:, g] = p @ v, p @ v.abs()
        grown += p.sum(0)
    return out, score[:n].double() + grown, size, grown


def pair_error(dtype, rows, D):
    """(of a weight, of the row's largest weight)"""
    if dtype is torch.bfloat16:
        return 2.0 ** -15, 0.0
    return 2.0 ** -22, 2.0 ** (-36 if rows > 16 and D > 128 else -48)


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("Sq,G,N,D", [(1, 1, 32769, 64), (1, 8, 131072, 128), (1, 16, 40001, 256),
                                      (4, 8, 32769, 128), (32, 4, 65536, 64), (1, 20, 1 << 20, 64),
                                      (2, 16, 40001, 256)])
def test_tail_beside_a_dominant_key(cuda_device, dtype, Sq, G, N, D):
    """The first key's logit is 18 above all others (weights 2^-26 of its own and a little
    either side); its value is 0 and theirs have one sign, so that the output is the tail's."""
    gen = torch.Generator(device="cuda").manual_seed(N + D)
    q = torch.zeros((1, Sq, G, D), dtype=dtype, device="cuda")
    q[..., 0] = 8.0
    k = torch.zeros((1, 1, N, D), dtype=dtype, device="cuda")
    # products of one element: the logits are exact, 0 but for a spread of 1 / 8 steps up to 1
    k[0, 0, :, 0] = torch.randint(0, 9, (N,), generator=gen, device="cuda").to(dtype) / 8
    k[0, 0, 0, 0] = 19.0
    v = (torch.rand((1, 1, N, D), generator=gen, device="cuda") + 0.5).to(dtype)
    v[0, 0, 0] = 0
    score = torch.zeros((1, 1, N), device="cuda")
    n = torch.tensor([N], dtype=torch.int32, device="cuda")
    out = L.attend_accumulate(q, k, v, n, score, scale=0.125)
    o, s, size, grown = reference(q[0], k[0, 0], v[0, 0], N, torch.zeros_like(score[0, 0]), 0.125)
    of_own, of_top = pair_error(dtype, Sq * G, D)
    rel = (3 * 19 + 64) * 2.0 ** -24 + of_own + N / 16 * 2.0 ** -23
    tol = rel * size + N * of_top * 1.5 + R.UNIT[dtype] * 1.01 * o.abs() + 2.0 ** -25
    assert ((out[0].double() - o).abs() <= tol).all(), ((out[0].double() - o).abs() / size).max()
    assert ((score[0, 0].double() - s).abs() <= ((3 * 19 + 64 + Sq * G) * 2.0 ** -24 + 2.0 ** -22) * s).all()


@pytest.mark.parametrize("Sq,Hq,Hkv,N,D", [(1, 8, 2, 30000, 128), (20, 4, 2, 24000, 64), (33, 8, 1, 9000, 128),
                                           (5, 12, 1, 7000, 256), (3, 2, 2, 40000, 16)])
def test_long_runs_in_fp16(cuda_device, Sq, Hq, Hkv, N, D):
    """Many key tiles to a block, with a peak in the middle that raises the references late."""
    gen = torch.Generator().manual_seed(N)
    B, G = 2, Hq // Hkv
    q = (torch.randn((B, Sq, Hq, D), generator=gen) * 1.5).half().cuda()
    k, v = (torch.randn((B, Hkv, N, D), generator=gen).half().cuda() for _ in range(2))
    k[:, :, N // 2] = (q[:, 0, 0] * 3)[:, None]
    score = torch.rand((B, Hkv, N), generator=gen).cuda()
    n = [N, N - 333]
    s = score.clone()
    out = L.attend_accumulate(q, k, v, torch.tensor(n, dtype=torch.int32, device="cuda"), s)
    reach = float(q.abs().max() * k.abs().max()) * D ** 0.5
    of_own, of_top = pair_error(torch.float16, Sq * G, D)
    # sums of D products average to a tenth of reach
    rel = (D * reach / 10 + 3 * reach + 64) * 2.0 ** -24
    for b in range(B):
        for h in range(Hkv):
            o, want, size, grown = reference(q[b, :, h * G:(h + 1) * G], k[b, h], v[b, h], n[b], score[b, h],
                                             D ** -0.5)
            off = (s[b, h, :n[b]].double() - want).abs()
            assert (off <= rel * grown + 2.0 ** -23 * want + Sq * G * 2.0 ** -126).all()
            tol = (rel + of_own + n[b] / 16 * 2.0 ** -23) * size + n[b] * of_top * float(v.abs().max()) + \
                R.UNIT[torch.float16] * 1.01 * o.abs() + 2.0 ** -25
            assert ((out[b, :, h * G:(h + 1) * G].double() - o).abs() <= tol).all()
        assert torch.equal(s[b, :, n[b]:], score[b, :, n[b]:])


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("step", [0.5, 2.7, 3.3, 9.0, 40.0])
@pytest.mark.parametrize("Sq,G,D", [(1, 4, 64), (9, 8, 128), (3, 8, 192)])
def test_logits_that_rise(cuda_device, dtype, step, Sq, G, D):
    """Each tile of 128 keys lies `step` above the one before: references are raised at every
    tile, at some, or late, and the largest weights come near the types' ends."""
    N = 128 * 12 + 37
    gen = torch.Generator(device="cuda").manual_seed(int(step * 10) + D)
    q = torch.zeros((1, Sq, G, D), dtype=dtype, device="cuda")
    q[..., 0] = 1.0
    q[..., 1] = torch.randn((1, Sq, G), generator=gen, device="cuda").to(dtype)
    k = torch.zeros((1, 1, N, D), dtype=dtype, device="cuda")
    k[0, 0, :, 0] = (torch.arange(N, device="cuda") // 128 * step).to(dtype)
    k[0, 0, :, 1] = torch.randn(N, generator=gen, device="cuda").to(dtype)
    v = torch.randn((1, 1, N, D), generator=gen, device="cuda").to(dtype)
    score = torch.zeros((1, 1, N), device="cuda")
    n = torch.tensor([N], dtype=torch.int32, device="cuda")
    out = L.attend_accumulate(q, k, v, n, score, scale=1.0)
    o, s, size, grown = reference(q[0], k[0, 0], v[0, 0], N, torch.zeros_like(score[0, 0]), 1.0)
    of_own, of_top = pair_error(dtype, Sq * G, D)
    reach = 12 * step + 20
    rel = (5 * reach + 64) * 2.0 ** -24
    tol = (rel + of_own + N / 16 * 2.0 ** -23) * size + N * of_top * float(v.abs().max()) + \
        R.UNIT[dtype] * 1.01 * o.abs() + 2.0 ** -25
    assert ((out[0].double() - o).abs() <= tol).all()
    assert ((score[0, 0].double() - s).abs() <= rel * s + 2.0 ** -22 * s + Sq * G * 2.0 ** -126).all()
