"""Plain 64-bit forms of the routing, expert-row, cache-attention and eviction
operators, row by row from their definitions, and the rounding units that the
tests' tolerances count.  Nothing here shares code with the library."""
import math

import numpy as np
import torch

# half a step relative to the value: the most that one rounding is off
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11,
        torch.float64: 2.0 ** -53}


def route_row(l, k, score="softmax", bias=None, groups=1, top_groups=None, group_top=2,
              renormalize=True, scale=1.0):
    """(weights, experts, scores) of one row of float64 logits."""
    E = l.size
    w, idx = np.zeros(k), np.full(k, -1, dtype=np.int64)
    if np.isnan(l).any() or (l == np.inf).any():
        return w + np.nan, idx, None
    live = l > -np.inf
    with np.errstate(over="ignore"):
        if score == "softmax":
            e = np.where(live, np.exp(np.where(live, l - (l[live].max() if live.any() else 0), 0)), 0)
            s = e / e.sum() if live.any() else e
        else:
            s = np.where(live, 1.0 / (1.0 + np.exp(-l)), 0.0)
    key = s.copy() if bias is None else s + bias
    if np.isnan(key[live]).any() or (key[live] == np.inf).any():
        return w + np.nan, idx, None
    key[~live] = -np.inf
    allowed = live & (key > -np.inf)
    top_groups = groups if top_groups is None else top_groups
    if top_groups < groups:
        size, value = E // groups, []
        for g in range(groups):
            mine = sorted((key[i] for i in range(g * size, (g + 1) * size) if allowed[i]),
                          reverse=True)[:group_top]
            value.append(sum(mine) if mine else -math.inf)
        kept = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
        for g in range(groups):
            if g not in kept:
                allowed[g * size:(g + 1) * size] = False
    order = l if bias is None else key  # the score rises strictly with the logit
    chosen = sorted((i for i in range(E) if allowed[i]), key=lambda i: (-order[i], i))[:k]
    idx[:len(chosen)] = chosen
    if renormalize and chosen:
        if score == "softmax":
            e = np.exp(l[chosen] - l[chosen].max())
        else:  # log sigmoid, shifted
            u = np.minimum(l[chosen], 0) - np.log1p(np.exp(-np.abs(l[chosen])))
            e = np.exp(u - u.max())
        w[:len(chosen)] = e / e.sum() * scale
    else:
        w[:len(chosen)] = s[chosen] * scale
    return w, idx, s


def route_grad_row(l, idx, u, score, renormalize, scale):
    """dL/dl of L = sum_j u_j w_j with the choice idx held fixed."""
    x = torch.tensor(l, dtype=torch.float64, requires_grad=True)
    on = [j for j in range(len(idx)) if idx[j] >= 0]
    if not on:
        return np.zeros_like(l)
    c = torch.tensor([int(idx[j]) for j in on])
    if renormalize:  # in logarithms: the ratio of scores that underflow is still one
        logs = torch.log_softmax(x, 0) if score == "softmax" else torch.nn.functional.logsigmoid(x)
        w = torch.softmax(logs[c], 0) * scale
    else:
        w = (torch.softmax(x, 0) if score == "softmax" else torch.sigmoid(x))[c] * scale
    (w * torch.tensor([u[j] for j in on], dtype=torch.float64)).sum().backward()
    return torch.nan_to_num(x.grad).numpy()


def plan(experts, E):
    """(offsets, slots, order) of the stable sort by expert; dropped ones last."""
    flat = experts.reshape(-1)
    where = [[] for _ in range(E + 1)]
    for i, e in enumerate(flat):
        where[e if 0 <= e < E else E].append(i)
    order = np.array([i for b in where for i in b], dtype=np.int64)
    slots = np.empty(flat.size, dtype=np.int64)
    slots[order] = np.arange(flat.size)
    offsets = np.cumsum([0] + [len(b) for b in where[:E]])
    return offsets, slots.reshape(experts.shape), order


def attend(q, k, v, lengths, score, scale):
    """(out, score) in float64; q (B, Sq, Hq, D), k and v (B, Hkv, N, D)."""
    B, Sq, Hq, D = q.shape
    Hkv, N = k.shape[1], k.shape[2]
    G = Hq // Hkv
    out, score = np.zeros(q.shape), score.astype(np.float64).copy()
    for b in range(B):
        n = min(max(int(lengths[b]), 0), N)
        for i in range(Sq):
            see = max(0, n - Sq + i + 1)
            if see == 0:
                continue
            for hq in range(Hq):
                h = hq // G
                x = (k[b, h, :see] @ q[b, i, hq]) * scale
                e = np.exp(x - x.max())
                p = e / e.sum()
                out[b, i, hq] = p @ v[b, h, :see]
                score[b, h, :see] += p
    return out, score


def evict_positions(score, n, budget, first, last):
    """Kept positions of one row, ascending."""
    if n <= budget:
        return np.arange(n)
    held = [i for i in range(n) if i < first or i >= n - last]
    free = [i for i in range(n) if first <= i < n - last]
    value = np.where(np.isnan(score), -np.inf, score.astype(np.float64))
    nan = np.isnan(score)
    free.sort(key=lambda i: (bool(nan[i]), -value[i], i))
    return np.array(sorted(held + free[:budget - len(held)]), dtype=np.int64)
