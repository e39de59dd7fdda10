"""Eviction into a caller's tensors: pieces that share memory are refused, pieces that lie side by
side are filled."""
import pytest
import torch

import sparse_selection_primitive_b200 as L
from tests.test_gpu_cache import check_evict, evict_inputs

pytestmark = pytest.mark.gpu
B, H, N, D, BUDGET = 2, 3, 200, 16, 40


def test_shared_pieces_are_refused(cuda_device):
    k, v, s = evict_inputs(1, B, H, N, D, torch.float32)
    n = torch.tensor([N, N], dtype=torch.int32).cuda()
    room = torch.zeros((B, H, BUDGET + 1, D), device="cuda")
    other, so = torch.zeros_like(room), torch.zeros((B, H, BUDGET), device="cuda")
    rows = room[:, :, :BUDGET]
    for out in ((rows, rows, so), (rows, room[:, :, 1:], so),
                (rows, room.view(-1)[8:8 + B * H * BUDGET * D].view(B, H, BUDGET, D), so),
                (rows, other, room.view(-1)[:B * H * BUDGET].view(B, H, BUDGET)),
                (other, rows, room.view(-1)[100:100 + B * H * BUDGET].view(B, H, BUDGET))):
        with pytest.raises(ValueError, match="share"):
            L.evict(k, v, s, n, BUDGET, out=out)


def test_pieces_side_by_side(cuda_device):
    for dtype in (torch.float32, torch.bfloat16):
        k, v, s = evict_inputs(2, B, H, N, D, dtype)
        want = L.evict(k, v, s, torch.tensor([N, 30], dtype=torch.int32).cuda(), BUDGET, first=2, last=4)
        so = torch.zeros((B, H, BUDGET), device="cuda")
        by_turns = torch.zeros((B, H, BUDGET, 2, D), dtype=dtype, device="cuda")
        halves = torch.zeros((B, H, 2 * BUDGET, D), dtype=dtype, device="cuda")
        for ko, vo in ((by_turns[:, :, :, 0], by_turns[:, :, :, 1]),
                       (halves[:, :, :BUDGET], halves[:, :, BUDGET:]),
                       (halves, halves[:, :, BUDGET:])):   # only the first rows are written
            e = check_evict(k, v, s, [N, 30], BUDGET, 2, 4, out=(ko, vo, so))
            assert torch.equal(e.k[:, :, :BUDGET], want.k) and torch.equal(e.v, want.v)
