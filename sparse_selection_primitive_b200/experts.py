"""Expert routing and the rows that follow it: ``route_experts`` (hard top-k of a
router's scores with differentiable weights), ``expert_plan`` (a stable sort of
the assignments by expert), ``expert_gather`` and ``expert_combine`` (rows to the
experts and their weighted sum back), each with its gradient.

The definitions stand in ``include/lapsum.h``; mixture-of-experts routing is one
of the uses the pages of "Fast LapSum: Exact Differentiable Top-k at Million
Scale" name (gist.science explainer pages, section 4.2).
"""
from __future__ import annotations

from typing import NamedTuple

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from ._launch import DTYPES, launch, need, no_tangents

SCORES = {"softmax": 0, "sigmoid": 1}


def _rows(x: torch.Tensor) -> torch.Tensor:
    """x with consecutive elements in each row and rows that do not overlap."""
    if x.stride(1) != 1 and x.shape[1] > 1 or x.shape[0] > 1 and x.stride(0) < x.shape[1]:
        return x.contiguous()
    return x


def _ld(x: torch.Tensor) -> int:
    return x.stride(0) if x.shape[0] > 1 else x.shape[1]


def _route(logits, k, score, bias, groups, top_groups, group_top, renormalize, scale):
    T, E = logits.shape
    weights = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    experts = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    if T > 0:
        launch(_lib().lapsum_route, logits.device, logits.data_ptr(), DTYPES[logits.dtype],
               _ld(logits), T, E, k, score, bias.data_ptr() if bias is not None else None, groups,
               top_groups, group_top, renormalize, scale, weights.data_ptr(), experts.data_ptr())
    return weights, experts


def route_backward(logits: torch.Tensor, weights: torch.Tensor, experts: torch.Tensor,
                   dweights: torch.Tensor, score: str = "softmax", renormalize: bool = True,
                   scale: float = 1.0) -> torch.Tensor:
    """The gradient of the logits from that of the weights, for the weights and
    experts that ``route_experts`` gave with the same score, renormalize and scale."""
    need(logits, "logits", DTYPES, 2)
    need(weights, "weights", (torch.float32,), 2, logits.device)
    need(experts, "experts", (torch.int32,), 2, logits.device)
    need(dweights, "dweights", (torch.float32,), 2, logits.device)
    if weights.shape != experts.shape or dweights.shape != experts.shape or \
            experts.shape[0] != logits.shape[0]:
        raise ValueError("weights, experts and dweights must be (rows of logits) x k")
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}")
    no_tangents("route_backward", logits, weights, dweights)
    return _route_grad(_rows(logits), weights.contiguous(), experts.contiguous(),
                       dweights.contiguous(), SCORES[score], bool(renormalize), float(scale))


def _once(backward):
    """once_differentiable, without its cost in a plain backward pass (no create_graph)."""
    checked = once_differentiable(backward)

    def run(ctx, *grads):
        return (checked if torch.is_grad_enabled() else backward)(ctx, *grads)
    return staticmethod(run)


def _route_grad(logits, weights, experts, dweights, score, renormalize, scale):
    T, E = logits.shape
    out = logits.new_empty((T, E))
    if T > 0:
        launch(_lib().lapsum_route_backward, logits.device, logits.data_ptr(),
               DTYPES[logits.dtype], _ld(logits), T, E, experts.shape[1], score, renormalize,
               scale, weights.data_ptr(), experts.data_ptr(), dweights.data_ptr(), out.data_ptr(),
               E)
    return out


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, score, bias, groups, top_groups, group_top, renormalize, scale):
        weights, experts = _route(logits, k, score, bias, groups, top_groups, group_top,
                                  renormalize, scale)
        ctx.save_for_backward(logits, weights, experts)
        ctx.how = (score, renormalize, scale)
        ctx.mark_non_differentiable(experts)
        ctx.set_materialize_grads(False)
        return weights, experts

    @_once
    def backward(ctx, dweights, _):
        if dweights is None:
            return (None,) * 9
        logits, weights, experts = ctx.saved_tensors
        return (_route_grad(logits, weights, experts, dweights.contiguous(), *ctx.how),
                None, None, None, None, None, None, None, None)


def route_experts(logits: torch.Tensor, k: int, *, score: str = "softmax", bias=None,
                  groups: int = 1, top_groups: int = None, group_top: int = 2,
                  renormalize: bool = True, scale: float = 1.0):
    """(weights, experts), both (T, k), of the k experts with the largest keys per row.

    ``logits`` (T, E) float32, bfloat16 or float16, E <= 1024; k and ``groups`` are at most
    32.  The scores are a ``softmax`` over the row or each logit's ``sigmoid``; ``bias`` (E,
    float32) is added for the choice only and gets no gradient.  With ``top_groups`` < ``groups``
    the choice is limited to the groups whose ``group_top`` (1 or 2) largest keys have
    the largest sum.  The weights (float32, differentiable in the logits) are the chosen
    scores, by default divided by their sum, times ``scale``.  Equal keys go to the
    lower index.  Logits of -inf are never chosen: places that find no expert hold
    expert -1 and weight 0.  A row with a NaN or +inf holds -1 and NaN."""
    need(logits, "logits", DTYPES, 2)
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}")
    k, groups, group_top = int(k), int(groups), int(group_top)
    top_groups = groups if top_groups is None else int(top_groups)
    if k < 1 or logits.shape[1] < 1:
        raise ValueError("k and the number of experts must be at least 1")
    if bias is not None:
        need(bias, "bias", (torch.float32,), 1, logits.device)
        if bias.shape[0] != logits.shape[1]:
            raise ValueError("bias must have one entry per expert")
        bias = bias.detach().contiguous()
    no_tangents("route_experts", logits)
    logits = _rows(logits)
    renormalize, scale = bool(renormalize), float(scale)
    run = _Route.apply if logits.requires_grad and torch.is_grad_enabled() else _route
    return run(logits, k, SCORES[score], bias, groups, top_groups, group_top, renormalize, scale)


class ExpertPlan(NamedTuple):
    """Where each of the T x k assignments goes: ``offsets`` (E + 1) each expert's first
    place and, last, the number of assignments that have an expert; ``slots`` (T, k) the
    place of an assignment; ``order`` (T k) the assignment t k + j of a place.  int32."""
    offsets: torch.Tensor
    slots: torch.Tensor
    order: torch.Tensor

    @property
    def live(self) -> int:
        """Address of the number of places in use."""
        return self.offsets.data_ptr() + 4 * (self.offsets.shape[0] - 1)


def expert_plan(experts: torch.Tensor, num_experts: int) -> ExpertPlan:
    """Sorts the assignments ``experts`` (T, k, int32) by expert, stably.  Values outside
    [0, num_experts) are dropped assignments; their places come behind all others."""
    need(experts, "experts", (torch.int32,), 2)
    experts = experts.contiguous()
    E, N, dev = int(num_experts), experts.numel(), experts.device
    if E < 1:
        raise ValueError("num_experts must be at least 1")
    if N == 0:
        return ExpertPlan(torch.zeros(E + 1, dtype=torch.int32, device=dev),
                          torch.empty_like(experts), experts.new_empty(0))
    nbytes = _lib().lapsum_expert_plan_workspace_bytes(N, E)
    # one piece of memory: the workspace (whole int32, aligned as the piece is), then the plan
    ws, offsets, order, slots = experts.new_empty(nbytes // 4 + E + 1 + 2 * N).split(
        (nbytes // 4, E + 1, N, N))
    launch(_lib().lapsum_expert_plan, dev, experts.data_ptr(), N, E, offsets.data_ptr(),
           slots.data_ptr(), order.data_ptr(), ws.data_ptr(), nbytes)
    return ExpertPlan(offsets, slots.view(experts.shape), order)


def _check_plan(plan: ExpertPlan, device):
    need(plan.offsets, "plan.offsets", (torch.int32,), 1, device)
    need(plan.slots, "plan.slots", (torch.int32,), 2, device)
    if not plan.slots.is_contiguous() or not plan.offsets.is_contiguous():
        raise ValueError("the plan's tensors must be contiguous")
    if plan.offsets.shape[0] < 2:  # the last entry is read
        raise ValueError("plan.offsets must have one entry more than there are experts")


def _gather(x, plan):
    (T, H), k = x.shape, plan.slots.shape[1]
    xs = x.new_empty((T * k, H))
    if xs.numel() > 0:
        launch(_lib().lapsum_expert_gather, x.device, x.data_ptr(), DTYPES[x.dtype], _ld(x), T, k,
               H, plan.slots.data_ptr(), plan.live, xs.data_ptr())
    return xs


def _combine(y, weights, plan):
    (T, k), H = plan.slots.shape, y.shape[1]
    out = y.new_empty((T, H))
    if y.numel() == 0:
        return out.zero_()
    launch(_lib().lapsum_expert_combine, y.device, y.data_ptr(), DTYPES[y.dtype], T, k, H,
           plan.slots.data_ptr(), plan.live, weights.data_ptr() if weights is not None else None,
           out.data_ptr())
    return out


class _Gather(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, offsets, slots, order):
        plan = ExpertPlan(offsets, slots, order)
        ctx.save_for_backward(offsets, slots)
        return _gather(x, plan)

    @_once
    def backward(ctx, dxs):
        offsets, slots = ctx.saved_tensors
        return _combine(dxs.contiguous(), None, ExpertPlan(offsets, slots, None)), None, None, None


def expert_gather(x: torch.Tensor, plan: ExpertPlan) -> torch.Tensor:
    """The rows of x (T, H) in expert order, (T k, H): row plan.slots[t, j] is x[t].
    Rows behind the last expert's are 0.  Differentiable in x."""
    need(x, "x", DTYPES, 2)
    _check_plan(plan, x.device)
    if x.shape[0] != plan.slots.shape[0]:
        raise ValueError("x must have one row per row of the plan")
    no_tangents("expert_gather", x)
    x = _rows(x)
    if x.requires_grad and torch.is_grad_enabled():
        return _Gather.apply(x, *plan)
    return _gather(x, plan)


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, offsets, slots):
        # y is needed for the weights' gradient only
        ctx.save_for_backward(y if ctx.needs_input_grad[1] else None, weights, offsets, slots)
        ctx.rows = y.shape
        return _combine(y, weights, ExpertPlan(offsets, slots, None))

    @_once
    def backward(ctx, dout):
        y, weights, offsets, slots = ctx.saved_tensors
        plan = ExpertPlan(offsets, slots, None)
        dout = _rows(dout)
        (T, k), H = slots.shape, dout.shape[1]
        dy = dout.new_empty(ctx.rows) if ctx.needs_input_grad[0] else None
        dw = torch.empty_like(weights) if ctx.needs_input_grad[1] else None
        if ctx.rows.numel() == 0:
            return dy, None if dw is None else dw.zero_(), None, None
        ptr = lambda x: None if x is None else x.data_ptr()  # noqa: E731
        launch(_lib().lapsum_expert_combine_backward_part, dout.device, dout.data_ptr(),
               DTYPES[dout.dtype], _ld(dout), ptr(y), T, k, H, slots.data_ptr(), plan.live,
               weights.data_ptr(), ptr(dy), ptr(dw))
        return dy, dw, None, None


def expert_combine(y: torch.Tensor, weights: torch.Tensor, plan: ExpertPlan) -> torch.Tensor:
    """(T, H): row t is the sum over j of weights[t, j] y[plan.slots[t, j]], in float32
    and rounded once to y's type; dropped assignments add nothing.  y (T k, H) holds
    the experts' results in the plan's order; weights (T, k) is float32.
    Differentiable in y and weights."""
    need(y, "y", DTYPES, 2)
    need(weights, "weights", (torch.float32,), 2, y.device)
    _check_plan(plan, y.device)
    if weights.shape != plan.slots.shape:
        raise ValueError("weights must have the shape of plan.slots")
    if y.shape[0] != plan.slots.numel():
        raise ValueError("y must have one row per assignment of the plan")
    no_tangents("expert_combine", y, weights)
    y, weights = y.contiguous(), weights.contiguous()
    if torch.is_grad_enabled() and (y.requires_grad or weights.requires_grad):
        return _Combine.apply(y, weights, plan.offsets, plan.slots)
    return _combine(y, weights, plan)
