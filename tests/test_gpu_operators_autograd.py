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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,k,H", [(9, 3, 40), (300, 8, 257), (70, 2, 2048), (1, 1, 1)])
def test_combination_forms_the_gradients_that_are_asked_for(cuda_device, dtype, T, k, H):
    """One of the two alone has the bits that it has beside the other."""
    gen = torch.Generator().manual_seed(T + H)
    experts = torch.randint(-1, 5, (T, k), generator=gen).to(torch.int32).cuda()
    plan = L.expert_plan(experts, 5)
    y0 = torch.randn((T * k, H), generator=gen).to(dtype).cuda()
    w0 = torch.rand((T, k), generator=gen).cuda()
    dout = torch.randn((T, H), generator=gen).to(dtype).cuda()

    def grads(wants_y, wants_w):
        y, w = y0.clone().requires_grad_(wants_y), w0.clone().requires_grad_(wants_w)
        out = L.expert_combine(y, w, plan)
        if not wants_w:
            y.detach().fill_(float("nan"))  # not kept, not read
        return torch.autograd.grad(out, [x for x in (y, w) if x.requires_grad], dout)

    dy, dw = grads(True, True)
    only_y, = grads(True, False)
    only_w, = grads(False, True)
    assert torch.equal(only_y, dy) and torch.equal(only_w, dw)
    # asked for one of two
    y, w = y0.clone().requires_grad_(True), w0.clone().requires_grad_(True)
    out = L.expert_combine(y, w, plan)
    assert torch.equal(torch.autograd.grad(out, y, dout, retain_graph=True)[0], dy)
    assert torch.equal(torch.autograd.grad(out, w, dout)[0], dw)


def test_combination_takes_no_memory_for_other_gradients(cuda_device):
    T, k, H = 4096, 8, 1024
    plan = L.expert_plan(torch.randint(0, 16, (T, k), dtype=torch.int32, device="cuda"), 16)
    w0, dout = torch.rand((T, k), device="cuda"), torch.randn((T, H), device="cuda")
    rows = T * k * H * 4

    def peak(wants_y, wants_w):
        y = torch.randn((T * k, H), device="cuda").requires_grad_(wants_y)
        w = w0.clone().requires_grad_(wants_w)
        out = L.expert_combine(y, w, plan)
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        torch.autograd.grad(out, y if wants_y else w, dout)
        return torch.cuda.max_memory_allocated() - before

    assert peak(True, False) >= rows
    assert peak(False, True) < rows / 8
    # a temporary y is not kept for the weights of a fixed router
    leaf = torch.randn((1, H), device="cuda", requires_grad=True)
    before = torch.cuda.memory_allocated()
    out = L.expert_combine(leaf.expand(T * k, H) * 1.0, w0, plan)
    assert torch.cuda.memory_allocated() - before < rows / 2
    assert out.grad_fn is not None


def test_tensors_that_a_graph_kept_are_seen_to_change(cuda_device):
    """Written in place, as by torch's own in-place operations: a backward pass that needs the
    values from before raises instead of taking the new ones."""
    gen = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(s, generator=gen).to(torch.bfloat16).cuda()
               for s in ((1, 1, 4, 16), (1, 2, 50, 16), (1, 2, 50, 16)))
    n = torch.tensor([50], dtype=torch.int32).cuda()

    def attend(**o):
        return lambda x: L.attend_accumulate(q, k, v, n, **{name: x for name in o["into"]},
                                             **({} if "score" in o["into"] else {"score": torch.zeros((1, 2, 50), device="cuda")}))

    def evict(at):
        def call(x):
            out = [torch.zeros((1, 2, 8, 16), dtype=torch.bfloat16, device="cuda"),
                   torch.zeros((1, 2, 8, 16), dtype=torch.bfloat16, device="cuda"),
                   torch.zeros((1, 2, 8), device="cuda")]
            out[at] = x
            L.evict(k, v, torch.rand((1, 2, 50), device="cuda"), n, 8, out=tuple(out))
        return call

    rows = torch.zeros((1, 2, 8, 16), dtype=torch.bfloat16, device="cuda")
    for write, x in ((attend(into=("score",)), torch.zeros((1, 2, 50), device="cuda")),
                     (attend(into=("score_out",)), torch.zeros((1, 2, 50), device="cuda")),
                     (attend(into=("out",)), torch.zeros((1, 1, 4, 16), dtype=torch.bfloat16, device="cuda")),
                     (evict(0), rows.clone()), (evict(1), rows.clone()),
                     (evict(2), torch.zeros((1, 2, 8), device="cuda"))):
        w = torch.ones_like(x, requires_grad=True)
        z = (w * x).sum()
        before = x._version
        write(x)
        assert x._version > before
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            z.backward()
        z = (w * x).sum()
        z.backward()
        assert torch.equal(w.grad, x)
    # what is only read keeps its version; inference tensors have none
    score, into = torch.zeros((1, 2, 50), device="cuda"), torch.zeros((1, 2, 50), device="cuda")
    was = [t._version for t in (q, k, v, n, score)]
    L.attend_accumulate(q, k, v, n, score, score_out=into)
    L.evict(k, v, score, n, 8)
    assert was == [t._version for t in (q, k, v, n, score)]
    with torch.inference_mode():
        L.attend_accumulate(q, k, v, n, torch.zeros((1, 2, 50), device="cuda"))


def test_results_into_tensors_that_require_a_gradient_are_refused(cuda_device):
    """As torch's own out= arguments; without grad mode, or detached, they are filled."""
    q, k, v = (torch.randn(s).to(torch.bfloat16).cuda() for s in ((1, 1, 4, 16), (1, 2, 50, 16), (1, 2, 50, 16)))
    n, score = torch.tensor([50], dtype=torch.int32).cuda(), torch.rand((1, 2, 50), device="cuda")
    rooms = [torch.zeros((1, 2, 8, 16), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    rooms.append(torch.zeros((1, 2, 8), device="cuda"))

    def evict(at):
        return lambda x: L.evict(k, v, score, n, 8, out=tuple(x if i == at else r for i, r in enumerate(rooms)))

    for call, x in ((lambda x: L.attend_accumulate(q, k, v, n, score, score_out=x), torch.zeros_like(score)),
                    (lambda x: L.attend_accumulate(q, k, v, n, score, out=x), torch.zeros_like(q)),
                    (evict(0), rooms[0].clone()), (evict(1), rooms[1].clone()), (evict(2), rooms[2].clone())):
        leaf = x.requires_grad_(True)
        with pytest.raises(RuntimeError, match="no gradient"):
            call(leaf)
        with torch.no_grad():
            call(leaf)
        call(leaf.detach())
        with fw.dual_level(), torch.no_grad(), pytest.raises(NotImplementedError):
            call(fw.make_dual(leaf.detach(), torch.ones_like(leaf)))
