"""A cache that is pruned by the weight its keys received: ``attend_accumulate``
(attention over the cache that adds each key's weight to a score) and ``evict``
(the keys with the largest scores, gathered in order).

The definitions stand in ``include/lapsum.h``; memory selection is one of the
uses the pages of "Fast LapSum: Exact Differentiable Top-k at Million Scale"
name (gist.science explainer pages, section 4.2).
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import torch
from torch.autograd.graph import increment_version

from . import _lib
from ._launch import DTYPES, apart, distinct, launch, need, no_gradient, no_tangents, overlap

_HALF = (torch.bfloat16, torch.float16)
_F32, _I32 = (torch.float32,), (torch.int32,)
_Strides13, _Strides16 = ctypes.c_int64 * 13, ctypes.c_int64 * 16


def _check_caches(k, v, score, lengths, dtypes):
    need(k, "k", dtypes, 4)
    dev, shape = k.device, k.shape
    need(v, "v", (k.dtype,), 4, dev)
    need(score, "score", _F32, 3, dev)
    need(lengths, "lengths", _I32, 1, dev)
    if v.shape != shape or score.shape != shape[:3] or lengths.shape[0] != shape[0]:
        raise ValueError("k and v must be (B, H, N, D), score (B, H, N) and lengths (B)")
    ks, vs, ss = k.stride(), v.stride(), score.stride()
    if (ks[3] != 1 or vs[3] != 1) and shape[3] > 1 or ss[2] != 1 and shape[2] > 1:
        raise ValueError("k, v and score must be consecutive in their last dimension")
    if not lengths.is_contiguous():
        raise ValueError("lengths must be contiguous")
    return ks, vs, ss


@functools.lru_cache(maxsize=256)
def _attend_workspace_bytes(B, Sq, Hq, Hkv, N, D) -> int:
    return _lib().lapsum_attend_workspace_bytes(B, Sq, Hq, Hkv, N, D)


def attend_accumulate(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lengths: torch.Tensor,
                      score: torch.Tensor, *, scale: float = None, score_out: torch.Tensor = None,
                      out: torch.Tensor = None) -> torch.Tensor:
    """Attention of q (B, Sq, Hq, D) over caches k, v (B, Hkv, N, D), bfloat16 or
    float16, filled up to ``lengths`` (B, int32) with the Sq tokens' own keys last;
    returns (B, Sq, Hq, D).  ``score`` (B, Hkv, N, float32) grows in place by the weight
    that each key received from the Sq * Hq / Hkv queries of its head, or
    ``score_out`` gets the sum and ``score`` stays.

    A token i sees the keys before lengths - Sq + i + 1; one that sees none gets 0.  Values of
    seen keys are to be finite: a NaN among the Sq tokens' own may reach the tokens before it.
    ``scale`` is D ** -0.5 by default.  D is a multiple of 16 up to 256; the tensors may
    be strided views whose rows start on 16 bytes.  No gradient."""
    ks, vs, ss = _check_caches(k, v, score, lengths, _HALF)
    need(q, "q", (k.dtype,), 4, k.device)
    B, Sq, Hq, D = q.shape
    _, Hkv, N, _ = k.shape
    if q.requires_grad or k.requires_grad or v.requires_grad or score.requires_grad:
        no_gradient("attend_accumulate")
    no_tangents("attend_accumulate", q, k, v, score)
    qs = q.stride()
    if B != k.shape[0] or D != k.shape[3] or Hkv < 1 or Hq % Hkv != 0:
        raise ValueError("q must be (B, Sq, Hq, D) with Hq a multiple of the caches' heads")
    if D > 1 and qs[3] != 1:
        raise ValueError("q must be consecutive in its last dimension")
    if score_out is None:
        score_out, outs = score, ss
    else:
        need(score_out, "score_out", _F32, 3, k.device)
        if score_out.requires_grad:
            no_gradient("attend_accumulate")
        no_tangents("attend_accumulate", score_out)
        outs = score_out.stride()
        if score_out.shape != score.shape or N > 1 and outs[2] != 1:
            raise ValueError("score_out must have score's shape, consecutive in its last dimension")
        same = outs == ss and score_out.data_ptr() == score.data_ptr()
        if not same and overlap(score, score_out):
            raise ValueError("score_out must be score itself or not overlap it")
    if not distinct(score_out):
        raise ValueError("the scores written must not share memory")
    written = score_out
    if out is None:
        out = q.new_empty(q.shape)
    else:
        written = score_out, out
        need(out, "out", (q.dtype,), 4, q.device)
        if out.requires_grad:
            no_gradient("attend_accumulate")
        no_tangents("attend_accumulate", out)
        if out.shape != q.shape or not out.is_contiguous():
            raise ValueError("out must be contiguous and have q's shape")
        if any(overlap(out, x) for x in (q, k, v, score, score_out)):
            raise ValueError("out must not overlap the inputs")
    if Sq < 1 or Hq < 1 or D < 1:
        raise ValueError("q must hold at least one token, head and element")
    if B == 0:
        return out
    if N == 0:
        return out.zero_()
    strides = _Strides13(qs[0], qs[2], qs[1], ks[0], ks[1], ks[2], vs[0], vs[1], vs[2], ss[0],
                         ss[1], outs[0], outs[1])
    nbytes = _attend_workspace_bytes(B, Sq, Hq, Hkv, N, D)
    ws = q.new_empty(nbytes // 2)  # two bytes an element
    launch(_lib().lapsum_attend_accumulate, q.device, q.data_ptr(), k.data_ptr(), v.data_ptr(),
           DTYPES[q.dtype], lengths.data_ptr(), strides, B, Sq, Hq, Hkv, N, D,
           D ** -0.5 if scale is None else float(scale), score.data_ptr(), score_out.data_ptr(),
           out.data_ptr(), ws.data_ptr(), nbytes)
    increment_version(written)  # a graph that kept their values has to see that they changed
    return out


class Evicted(NamedTuple):
    """The caches and scores that stayed, their positions before (-1: none) and the
    new lengths."""
    k: torch.Tensor
    v: torch.Tensor
    score: torch.Tensor
    positions: torch.Tensor
    lengths: torch.Tensor


def evict(k: torch.Tensor, v: torch.Tensor, score: torch.Tensor, lengths: torch.Tensor,
          budget: int, *, first: int = 0, last: int = 0, out=None) -> Evicted:
    """Keeps ``budget`` of the first ``lengths`` (B, int32) rows of caches k, v
    (B, H, N, D; float32, bfloat16 or float16) per sequence and head: the first
    ``first``, the last ``last``, and those between with the largest ``score``
    (B, H, N, float32; ties: the lower position), in the order of their positions.

    ``out`` may hold the caches and scores to fill, (k, v, score) with at least
    ``budget`` rows, that share no memory with the inputs or with each other (k and v may lie
    side by side in one tensor); rows from ``budget`` on are left as they were.  Rows that no key
    fills (fewer than ``budget`` in the cache) are 0 and their positions -1."""
    ks, vs, ss = _check_caches(k, v, score, lengths, DTYPES)
    if k.requires_grad or v.requires_grad or score.requires_grad:
        no_gradient("evict")
    no_tangents("evict", k, v, score)
    B, H, N, D = k.shape
    budget, first, last = int(budget), int(first), int(last)
    if budget < 1 or first < 0 or last < 0 or first + last > budget:
        raise ValueError("budget must be at least 1, and first + last at most budget")
    if out is None:
        ko = k.new_empty((B, H, budget, D))
        vo = torch.empty_like(ko)
        so = score.new_empty((B, H, budget))
    else:
        ko, vo, so = out
        need(ko, "out[0]", (k.dtype,), 4, k.device)
        need(vo, "out[1]", (k.dtype,), 4, k.device)
        need(so, "out[2]", (torch.float32,), 3, k.device)
        if ko.requires_grad or vo.requires_grad or so.requires_grad:
            no_gradient("evict")
        no_tangents("evict", ko, vo, so)
        for x, d in ((ko, (D,)), (vo, (D,)), (so, ())):
            if x.shape[:2] != (B, H) or x.shape[2] < budget or tuple(x.shape[3:]) != d or \
                    x.shape[-1] > 1 and x.stride(-1) != 1 or not distinct(x):
                raise ValueError("out must be (B, H, C, D), (B, H, C, D) and (B, H, C) with "
                                 "C >= budget, consecutive in the last dimension")
        if any(overlap(x, y) for x in (ko, vo, so) for y in (k, v, score, lengths)):
            raise ValueError("out must not overlap the inputs")
        kw, vw, sw = (x[:, :, :budget] for x in (ko, vo, so))  # what is written
        if not (apart(kw, vw) and apart(kw, sw) and apart(vw, sw)):
            raise ValueError("the tensors of out must not share memory")
    positions = lengths.new_empty((B, H, budget))
    left = torch.empty_like(lengths)
    result = Evicted(ko, vo, so, positions, left)
    if B * H * D == 0 or N == 0:
        if B * H > 0:
            raise ValueError("the caches must hold at least one row of one element")
        left.copy_(lengths.clamp(0, min(N, budget)))
        return result
    strides = _Strides16(*ks[:3], *vs[:3], *ss[:2], *ko.stride()[:3], *vo.stride()[:3],
                         *so.stride()[:2])
    launch(_lib().lapsum_evict, k.device, k.data_ptr(), v.data_ptr(), DTYPES[k.dtype],
           score.data_ptr(), lengths.data_ptr(), strides, B, H, N, D, budget, first, last,
           ko.data_ptr(), vo.data_ptr(), so.data_ptr(), positions.data_ptr(), left.data_ptr())
    if out is not None:
        increment_version((ko, vo, so))
    return result
