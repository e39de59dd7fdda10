"""What the routing, expert-row and cache calls do to autograd: forward-mode inputs are refused."""
import pytest
import torch
import torch.autograd.forward_ad as fw

import sparse_selection_primitive_b200 as L

pytestmark = pytest.mark.gpu


def layer():
    """Calls by name, each on a dict of its differentiable inputs."""
    gen = torch.Generator().manual_seed(3)
    logits = torch.randn((6, 16), generator=gen).cuda()
    w, idx = L.route_experts(logits, 4)
    plan = L.expert_plan(idx, 16)
    x, y = torch.randn((6, 32), generator=gen).cuda(), torch.randn((24, 32), generator=gen).cuda()
    q, k, v = (torch.randn(s, generator=gen).to(torch.bfloat16).cuda()
               for s in ((1, 1, 4, 16), (1, 2, 50, 16), (1, 2, 50, 16)))
    score, n = torch.rand((1, 2, 50), generator=gen).cuda(), torch.tensor([50], dtype=torch.int32).cuda()
    return [
        ("route_experts", dict(logits=logits), lambda logits: L.route_experts(logits, 4)),
        ("route_backward", dict(logits=logits, weights=w, dweights=torch.ones_like(w)),
         lambda logits, weights, dweights: L.route_backward(logits, weights, idx, dweights)),
        ("expert_gather", dict(x=x), lambda x: L.expert_gather(x, plan)),
        ("expert_combine", dict(y=y, weights=w), lambda y, weights: L.expert_combine(y, weights, plan)),
        ("attend_accumulate", dict(q=q, k=k, v=v, score=score),
         lambda q, k, v, score: L.attend_accumulate(q, k, v, n, score)),
        ("evict", dict(k=k, v=v, score=score), lambda k, v, score: L.evict(k, v, score, n, 8)),
    ]


def test_forward_mode_is_refused(cuda_device):
    """A tangent on any of the inputs, whether or not a gradient is asked for as well; inside a
    level without tangents the calls go on."""
    for name, inputs, call in layer():
        with fw.dual_level():
            call(**inputs)
            for which in inputs:
                for grad in (False, True):
                    base = inputs[which].detach().requires_grad_(grad)
                    dual = fw.make_dual(base, torch.ones_like(base))
                    with pytest.raises(RuntimeError):
                        call(**{**inputs, which: dual})
                    with torch.no_grad(), pytest.raises(NotImplementedError, match=name):
                        call(**{**inputs, which: dual})
        call(**inputs)


def test_jvp_is_refused(cuda_device):
    for name, inputs, call in layer():
        which, x = next(iter(inputs.items()))
        with pytest.raises(RuntimeError):
            torch.func.jvp(lambda t: call(**{**inputs, which: t}), (x,), (torch.ones_like(x),))
