"""Routing at the most experts a row can choose (32, a lane of a warp each), with a bias."""
import pytest
import torch

import sparse_selection_primitive_b200 as L
from tests.test_gpu_experts import check_route, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [32, 33, 64, 100, 257, 1024])
def test_choice(cuda_device, score, E):
    """Near and exact ties at every rank, the last one too, rows with fewer than 32 finite
    logits, and all logits equal."""
    bias = (torch.randn(E, generator=torch.Generator().manual_seed(E)) * 0.05).cuda()
    flat = torch.zeros(E, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        check_route(rows(E, 40, E, dtype), 32, score=score, bias=bias)
    check_route(rows(E + 1, 12, E, torch.float32).round(), 32, score=score, bias=flat)
    check_route(torch.zeros((3, E), device="cuda"), 32, score=score, bias=flat)
    # logits a few units apart: scores that round to the same fp32 value
    near = torch.full((16, E), 3.0) + torch.arange(E) * 2.0 ** -22
    near = near[:, torch.randperm(E, generator=torch.Generator().manual_seed(5))].cuda()
    check_route(near, 32, score=score, bias=flat)
    x = rows(E + 2, 6, E, torch.float32).clone()
    x[0, 5:] = -float("inf")
    x[1] = -float("inf")
    x[2, 31:] = -float("inf")
    check_route(x, 32, score=score, bias=bias)
    # the 32nd and 33rd keys alone are near: 32 clear ones, then two of nearly the same
    if E > 33:
        y = torch.full((4, E), -4.0)
        y[:, :31] = torch.arange(31) * 0.1
        y[:, 31] = -1.0
        y[:, 32] = torch.nextafter(torch.tensor(-1.0), torch.tensor(0.0))
        check_route(y.cuda(), 32, score=score, bias=flat)


def test_cost(cuda_device):
    """32 experts take the fast path as 31 do (in fp64 for every row they took 2.7 times as long)."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    l = torch.randn((16384, 256), device="cuda", generator=gen) * 1.5
    bias = torch.randn(256, device="cuda", generator=gen) * 0.05

    def micros(k):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(10):
                L.route_experts(l, k, score="sigmoid", bias=bias)
        best = float("inf")
        for _ in range(8):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            graph.replay()
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b) * 100)
        return best

    assert micros(32) <= 2 * micros(31)
