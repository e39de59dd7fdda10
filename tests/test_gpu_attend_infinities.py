"""Cache attention with infinities among a cache's own keys: a key whose logit is -inf for every
query takes no weight and adds nothing, whatever the number of rows is padded to."""
import pytest
import torch

import sparse_selection_primitive_b200 as L

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Sq,G", [(1, 1), (1, 2), (1, 3), (1, 5), (1, 8), (1, 15), (1, 16), (1, 17), (1, 40),
                                  (3, 7), (2, 64), (1, 130)])
def test_keys_of_no_weight(cuda_device, dtype, Sq, G):
    """Against the same call over a cache in which those keys' logits are finite and 200 below
    the others (weights e^-200: 0 in fp32), which gives the same bits."""
    B, H, N, D = 2, 2, 700, 64
    gen = torch.Generator().manual_seed(Sq * 100 + G)
    q = torch.randn((B, Sq, H * G, D), generator=gen)
    q[..., 5] = q[..., 5].abs() + 0.5       # times -inf: -inf for every query
    q = q.to(dtype).cuda()
    k, v = (torch.randn((B, H, N, D), generator=gen).to(dtype).cuda() for _ in range(2))
    score = torch.rand((B, H, N), generator=gen).cuda()
    n = torch.tensor([N, 433], dtype=torch.int32, device="cuda")
    hidden = torch.zeros(N, dtype=torch.bool, device="cuda")
    hidden[[0, 7, 130, 131, 400]] = True
    both = []
    for value in (-float("inf"), -6e4 if dtype is torch.float16 else -1e5):
        kk, s = k.clone(), score.clone()
        kk[:, :, hidden, 5] = value
        out = L.attend_accumulate(q, kk, v, n, s)
        assert not out.isnan().any()
        assert torch.equal(s[:, :, hidden], score[:, :, hidden])
        both.append((out, s))
    assert torch.equal(both[0][0], both[1][0]) and torch.equal(both[0][1], both[1][1])
