"""What is measured of the operators around hard selection: expert routing, the
movement of tokens to experts and back, attention over a cache that accumulates
each key's weight, and eviction from that cache.

A case names its operator in ``op``.  ``prepare`` makes the inputs on the GPU from
the seed, ``run`` makes one pass (the plain form in elementary torch operations, or
the library's calls where ``own`` is true), ``exact`` gives the same outputs from
the definitions in 64 bits, and ``work`` the bytes and operations that a pass
cannot do without.
"""
import math

import torch

own = False
device = "cuda"

_TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16, "float16": torch.float16}
_SIZE = {"float32": 4, "bfloat16": 2, "float16": 2}


def listed():
    return [
        # Routing.  One token of a serving step: sigmoid scores, a bias that balances the
        # load, eight groups of which four are kept; only latency counts.
        dict(name="route_one_token", op="route", T=1, E=256, k=8, score="sigmoid", bias=True,
             groups=8, top_groups=4, renormalize=True, scale=2.5, dtype="float32", train=False),
        # The router batch of this repository's workloads (16384 x 256, 8 of them), forward
        # and backward, with a softmax over all experts and renormalised weights.
        dict(name="route_train_16384x256", op="route", T=16384, E=256, k=8, score="softmax",
             bias=False, groups=1, top_groups=1, renormalize=True, scale=1.0, dtype="float32",
             train=True),
        # The same batch as grouped sigmoid routing with a bias, 16-bit logits.
        dict(name="route_grouped_bf16", op="route", T=16384, E=256, k=8, score="sigmoid",
             bias=True, groups=8, top_groups=4, renormalize=True, scale=2.5, dtype="bfloat16",
             train=True),
        # An odd batch over an odd number of experts; weights that are not renormalised, so
        # that the gradient reaches every expert.
        dict(name="route_odd_5003x100", op="route", T=5003, E=100, k=5, score="softmax", bias=False,
             groups=1, top_groups=1, renormalize=False, scale=1.0, dtype="float16", train=True),
        # Tokens to experts and back.  A serving step of 64 sequences.
        dict(name="experts_step_64x4096", op="experts", T=64, E=256, k=8, H=4096, drop=0.0,
             dtype="bfloat16", train=False),
        # A training batch, forward and backward: the largest rows moved.
        dict(name="experts_train_16384x2048", op="experts", T=16384, E=256, k=8, H=2048, drop=0.0,
             dtype="bfloat16", train=True),
        # Odd sizes in fp32, with a tenth of the assignments dropped.
        dict(name="experts_odd_1001x1000", op="experts", T=1001, E=37, k=3, H=1000, drop=0.1,
             dtype="float32", train=True),
        # Attention over a cache.  One sequence, one new token, an odd cache length.
        dict(name="attend_one_4099", op="attend", B=1, Hkv=8, G=4, Sq=1, D=128, N=4099,
             ragged=False, dtype="bfloat16"),
        # A serving batch with ragged lengths: 1 GB of keys and values.
        dict(name="attend_batch_32x8192", op="attend", B=32, Hkv=8, G=8, Sq=1, D=128, N=8192,
             ragged=True, dtype="bfloat16"),
        # The window of the last 32 queries of two long prompts, which ranks a prompt's keys
        # before the first eviction.
        dict(name="attend_window_2x32768", op="attend", B=2, Hkv=8, G=4, Sq=32, D=128, N=32768,
             ragged=False, dtype="bfloat16"),
        # Eviction.  One sequence's cache from an odd length to a quarter.
        dict(name="evict_one_4099", op="evict", B=1, Hkv=8, N=4099, budget=1024, first=4, last=64,
             D=128, ragged=False, dtype="bfloat16"),
        # The memory-selection batch of this repository's workloads: 256 rows of 65536 scores
        # with many ties, 1024 of them kept.
        dict(name="evict_batch_256x65536", op="evict", B=32, Hkv=8, N=65536, budget=1024, first=4,
             last=128, D=64, ragged=True, dtype="bfloat16"),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route", "experts", "attend", "attend", "evict"])
    dtype = rng.choice(["bfloat16", "float16", "float32"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * _spread(rng, 8, 512 // groups)
        return dict(op=op, T=_spread(rng, 1, 16384), E=E, k=rng.randint(1, min(E // groups, 12)),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups,
                    top_groups=rng.randint(1, groups), renormalize=rng.random() < 0.6,
                    scale=rng.choice([1.0, 2.5]), dtype=dtype, train=rng.random() < 0.7)
    if op == "experts":
        return dict(op=op, T=_spread(rng, 1, 8192), E=_spread(rng, 2, 384), k=rng.randint(1, 8),
                    H=8 * _spread(rng, 8, 256) + rng.choice([0, 0, 1, 4]),
                    drop=rng.choice([0.0, 0.0, 0.2]), dtype=dtype, train=rng.random() < 0.7)
    if op == "attend":
        Hkv, G, D = rng.choice([1, 2, 4, 8]), rng.randint(1, 12), rng.choice([64, 96, 128])
        N = _spread(rng, 1, 32768)
        Sq = min(N, rng.choice([1, 1, 1, _spread(rng, 2, 48)]))
        most = (1 << 28) // (N * Hkv * 128 * max(1, Sq * G // 16))
        return dict(op=op, B=_spread(rng, 1, max(1, min(32, most))), Hkv=Hkv, G=G, Sq=Sq, D=D, N=N,
                    ragged=rng.random() < 0.5, dtype=rng.choice(["bfloat16", "float16"]))
    Hkv, N = rng.choice([1, 2, 4, 8]), _spread(rng, 2, 65536)
    budget = _spread(rng, 1, N)
    first = min(4, budget // 4)
    return dict(op=op, B=_spread(rng, 1, max(1, min(32, (1 << 24) // (N * Hkv)))), Hkv=Hkv, N=N,
                budget=budget, first=first, last=min(64, budget // 2), D=rng.choice([64, 96, 128]),
                ragged=rng.random() < 0.5, dtype=dtype)


# --- inputs ----------------------------------------------------------------------------------
def _normal(gen, shape, dtype, scale=1.0):
    x = torch.empty(shape, dtype=dtype, device=device).normal_(generator=gen)
    return x if scale == 1.0 else x.mul_(scale)


def _lengths(case, gen):
    """One length a sequence: all of N, or spread from a quarter of it upwards."""
    B, N = case["B"], case["N"]
    if not case["ragged"]:
        return torch.full((B,), N, dtype=torch.int32, device=device)
    return torch.randint(max(1, N // 4), N + 1, (B,), generator=gen, device=device).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device=device).manual_seed(int(seed))
    s = dict(case)
    dt = _TYPES[case["dtype"]]
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = _normal(gen, (T, E), dt, 1.5)
        s["bias_t"] = _normal(gen, (E,), torch.float32, 0.05) if case["bias"] else None
        s["dw"] = _normal(gen, (T, k), torch.float32)
        s["x"] = s["logits"].clone().requires_grad_(True) if case["train"] else s["logits"]
    elif case["op"] == "experts":
        T, E, k, H = case["T"], case["E"], case["k"], case["H"]
        # each token's experts are different ones, and some experts are busier than others
        pull = _normal(gen, (1, E), torch.float32, 0.7)
        noise = _normal(gen, (T, max(E, k)), torch.float32)
        noise[:, :E] += pull
        experts = noise.argsort(1, descending=True)[:, :k].to(torch.int32)
        experts = torch.where(experts < E, experts, torch.full_like(experts, -1))
        if case["drop"] > 0:
            gone = torch.rand((T, k), generator=gen, device=device) < case["drop"]
            experts = torch.where(gone, torch.full_like(experts, -1), experts)
        s["experts"] = experts.contiguous()
        w = torch.rand((T, k), generator=gen, device=device) + 0.05
        s["w"] = w / w.sum(1, keepdim=True)
        s["x"] = _normal(gen, (T, H), dt)
        s["y"] = _normal(gen, (T * k, H), dt)
        if case["train"]:
            s["dxs"] = _normal(gen, (T * k, H), dt)
            s["dout"] = _normal(gen, (T, H), dt)
            for name in ("x", "y", "w"):
                s[name].requires_grad_(True)
    elif case["op"] == "attend":
        B, Hkv, G, Sq, D, N = (case[i] for i in ("B", "Hkv", "G", "Sq", "D", "N"))
        s["q"] = _normal(gen, (B, Sq, Hkv * G, D), dt, 1.5)
        s["kc"] = _normal(gen, (B, Hkv, N, D), dt)
        s["vc"] = _normal(gen, (B, Hkv, N, D), dt)
        s["lengths"] = _lengths(case, gen)
        inside = torch.arange(N, device=device) < s["lengths"][:, None, None]
        s["score"] = torch.rand((B, Hkv, N), generator=gen, device=device) * inside
        s["score_out"] = torch.zeros_like(s["score"])
    else:
        B, Hkv, D, N = (case[i] for i in ("B", "Hkv", "D", "N"))
        s["kc"] = _normal(gen, (B, Hkv, N, D), dt)
        s["vc"] = _normal(gen, (B, Hkv, N, D), dt)
        s["lengths"] = _lengths(case, gen)
        # accumulated weight is small for most keys and large for a few; multiples of 2^-12
        # make many exact ties among the small ones
        x = _normal(gen, (B, Hkv, N), torch.float32, 2.0)
        s["score"] = x.sub_(4.0).exp_().mul_(4096.0).round_().div_(4096.0)
    return s


# --- the plain forms -------------------------------------------------------------------------
def _plain_route(s):
    """Scores, keys and weights in 64 bits: two keys may lie nearer than 32 bits tell."""
    l = s["logits"].double()
    T, E = l.shape
    k, G = s["k"], s["groups"]
    if s["score"] == "softmax":
        e = (l - l.amax(1, keepdim=True)).exp()
        p = e / e.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + (-l).exp())
    key = p if s["bias_t"] is None else p + s["bias_t"].double()
    if G > 1:
        by_group = key.view(T, G, E // G)
        best = by_group.sort(dim=2, descending=True)[0][:, :, :2].sum(2)
        kept = best.sort(dim=1, descending=True, stable=True)[1][:, :s["top_groups"]]
        keep = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        key = torch.where(keep[:, :, None], by_group, -math.inf).view(T, E)
    idx = key.sort(dim=1, descending=True, stable=True)[1][:, :k]
    ps = p.gather(1, idx)
    total = ps.sum(1, keepdim=True) if s["renormalize"] else 1.0
    w = ps / total * s["scale"]
    out = [w.float(), idx.to(torch.int32)]
    if s["train"]:
        dw = s["dw"].double() * s["scale"]
        dp = (dw - (dw * ps / total).sum(1, keepdim=True)) / total if s["renormalize"] else dw
        full = torch.zeros_like(p).scatter_(1, idx, dp)
        if s["score"] == "softmax":
            dl = p * (full - (full * p).sum(1, keepdim=True))
        else:
            dl = full * p * (1.0 - p)
        out.append(dl.to(s["logits"].dtype))
    return out


def _plain_plan(experts, E):
    flat = experts.reshape(-1).long()
    flat = torch.where(flat < 0, E, flat)
    order = flat.sort(dim=0, stable=True)[1]
    slots = torch.empty_like(order).scatter_(0, order, torch.arange(order.numel(), device=flat.device))
    counts = torch.zeros(E + 1, dtype=torch.int64, device=flat.device)
    counts.scatter_add_(0, flat, torch.ones_like(flat))
    offsets = torch.cat([counts.new_zeros(1), counts[:E].cumsum(0)])
    return offsets.to(torch.int32), slots.view(experts.shape), order


def _plain_experts(s):
    with torch.no_grad():
        T, k, H = s["T"], s["k"], s["H"]
        x, y, w = s["x"], s["y"], s["w"]
        offsets, slots, order = _plain_plan(s["experts"], s["E"])
        used = (s["experts"] >= 0)
        of = order // k  # the token of each row
        row = used.reshape(-1)[order]
        xs = torch.where(row[:, None], x[of], torch.zeros((), dtype=x.dtype, device=x.device))
        wu = torch.where(used, w, 0.0)
        yt = torch.where(used[:, :, None], y[slots].float(), 0.0)  # (T, k, H)
        out = (wu[:, :, None] * yt).sum(1).to(x.dtype)
        got = [offsets, slots.to(torch.int32), order.to(torch.int32), xs, out]
        if s["train"]:
            dx = torch.where(used[:, :, None], s["dxs"][slots].float(), 0.0).sum(1).to(x.dtype)
            dout = s["dout"].float()
            dw = (dout[:, None, :] * yt).sum(2)
            dy = (torch.where(row, wu.reshape(-1)[order], 0.0)[:, None] * dout[of]).to(y.dtype)
            got += [dx, dy, dw]
        return got


def _plain_attend(s):
    B, Hkv, G, Sq, D, N = (s[i] for i in ("B", "Hkv", "G", "Sq", "D", "N"))
    q = s["q"].float().view(B, Sq, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, Sq * G, D)
    x = (q @ s["kc"].float().transpose(2, 3)) * D ** -0.5
    # query i of Sq sees the keys before length - Sq + i + 1
    upto = s["lengths"][:, None].long() - Sq + 1 + torch.arange(Sq, device=q.device)
    upto = upto.repeat_interleave(G, 1)[:, None, :, None]
    seen = torch.arange(N, device=q.device) < upto
    x = torch.where(seen, x, -math.inf)
    top = x.amax(3, keepdim=True)
    e = torch.where(seen, (x - torch.where(top > -math.inf, top, 0.0)).exp(), 0.0)
    total = e.sum(3, keepdim=True)
    p = e / torch.where(total > 0, total, 1.0)
    inside = torch.arange(N, device=q.device) < s["lengths"][:, None, None]
    v = torch.where(inside[..., None], s["vc"].float(), 0.0)
    out = (p @ v).view(B, Hkv, Sq, G, D).permute(0, 2, 1, 3, 4).reshape(B, Sq, Hkv * G, D)
    return [out.to(s["q"].dtype), s["score"] + p.sum(2)]


def _plain_evict(s):
    N, budget = s["N"], s["budget"]
    n = s["lengths"].long()[:, None, None]
    at = torch.arange(N, device=n.device)
    held = (at < s["first"]) | (at >= n - s["last"])
    key = torch.where(held, math.inf, s["score"])
    key = torch.where(at < n, key, -math.inf)
    pos = key.sort(dim=2, descending=True, stable=True)[1][:, :, :budget]
    pos = torch.where(pos < n, pos, N).sort(dim=2)[0]  # ascending, absent ones last
    real = pos < N
    src = torch.where(real, pos, 0)
    kept = lambda c: torch.where(real[..., None], c.gather(2, src[..., None].expand(-1, -1, -1, c.shape[3])), 0.0).to(c.dtype)  # noqa: E731
    score = torch.where(real, s["score"].gather(2, src), 0.0)
    left = torch.clamp(s["lengths"], max=budget).to(torch.int32)
    return [kept(s["kc"]), kept(s["vc"]), score, torch.where(real, pos, -1).to(torch.int32), left]


# --- the library's calls ---------------------------------------------------------------------
def _own_route(s):
    import sparse_selection_primitive_b200 as L
    w, idx = L.route_experts(s["x"], s["k"], score=s["score"], bias=s["bias_t"], groups=s["groups"],
                             top_groups=s["top_groups"], renormalize=s["renormalize"],
                             scale=s["scale"])
    if not s["train"]:
        return [w, idx]
    return [w, idx, torch.autograd.grad(w, s["x"], s["dw"])[0]]


def _own_experts(s):
    import sparse_selection_primitive_b200 as L
    plan = L.expert_plan(s["experts"], s["E"])
    xs = L.expert_gather(s["x"], plan)
    out = L.expert_combine(s["y"], s["w"], plan)
    got = [plan.offsets, plan.slots, plan.order, xs, out]
    if s["train"]:
        dx, = torch.autograd.grad(xs, s["x"], s["dxs"])
        dy, dw = torch.autograd.grad(out, (s["y"], s["w"]), s["dout"])
        got += [dx, dy, dw]
    return got


def _own_attend(s):
    import sparse_selection_primitive_b200 as L
    out = L.attend_accumulate(s["q"], s["kc"], s["vc"], s["lengths"], s["score"],
                              score_out=s["score_out"])
    return [out, s["score_out"]]


def _own_evict(s):
    import sparse_selection_primitive_b200 as L
    e = L.evict(s["kc"], s["vc"], s["score"], s["lengths"], s["budget"], first=s["first"],
                last=s["last"])
    return [e.k, e.v, e.score, e.positions, e.lengths]


def run(state):
    if own:
        return globals()["_own_" + state["op"]](state)
    return globals()["_plain_" + state["op"]](state)


# --- what a pass cannot do without -----------------------------------------------------------
def work(case):
    es = _SIZE[case["dtype"]]
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        moved = T * E * es + T * k * 8 + (T * E * es + T * k * 4 if case["train"] else 0)
        return {"bytes": moved + (4 * E if case["bias"] else 0),
                "flops": T * E * (12 if case["train"] else 8)}
    if case["op"] == "experts":
        T, k, H, E = case["T"], case["k"], case["H"], case["E"]
        N = T * k
        moved = 4 * N * 3 + 4 * (E + 1) + 4 * N + es * H * (T + N + N + T)
        flops = 2 * N * H
        if case["train"]:
            moved += es * H * (N + T + T + N) + 4 * N
            flops += 4 * N * H
        return {"bytes": moved, "flops": flops}
    n = (5 * case["N"] / 8 if case["ragged"] else case["N"]) * case["B"] * case["Hkv"]
    if case["op"] == "attend":
        G, Sq, D = case["G"], case["Sq"], case["D"]
        rows = case["B"] * case["Hkv"] * G * Sq
        return {"bytes": int(n * (2 * D * es + 8) + 2 * rows * D * es), "flops": int(4 * n * G * Sq * D)}
    kept = case["B"] * case["Hkv"] * min(case["budget"], case["N"])
    return {"bytes": int(4 * n + kept * (4 * case["D"] * es + 8)), "flops": int(2 * n)}


# --- the definitions in 64 bits --------------------------------------------------------------
def _exact_route(s):
    logits, k, G = s["logits"].detach().double(), s["k"], s["groups"]
    T, E = logits.shape
    w_all, i_all, d_all = [], [], []
    earlier = torch.arange(E, device=device)[None, :] < torch.arange(E, device=device)[:, None]
    size = E // G
    for a in range(0, T, 512):
        l = logits[a:a + 512].clone().requires_grad_(True)
        p = torch.softmax(l, 1) if s["score"] == "softmax" else torch.sigmoid(l)
        key = p.detach().clone()
        if s["bias_t"] is not None:
            key += s["bias_t"].double()
        t = key.shape[0]
        if G > 1:
            parts = key.view(t, G, size)
            hi = parts.max(2)
            rest = parts.scatter(2, hi[1][..., None], -math.inf)
            best = hi[0] + (rest.amax(2) if size > 1 else 0.0)
            ahead = (best[:, None, :] > best[:, :, None]) | (
                (best[:, None, :] == best[:, :, None]) & earlier[:G, :G])
            key = torch.where((ahead.sum(2) < s["top_groups"])[..., None], parts, -math.inf).reshape(t, E)
        # an expert's rank is the number of experts that come before it
        before = (key[:, None, :] > key[:, :, None]) | ((key[:, None, :] == key[:, :, None]) & earlier)
        rank = before.sum(2)
        idx = torch.empty((t, E), dtype=torch.int64, device=device)
        idx.scatter_(1, rank, torch.arange(E, device=device).expand(t, E))
        idx = idx[:, :k]
        w = p.gather(1, idx)
        if s["renormalize"]:
            w = w / w.sum(1, keepdim=True)
        w = w * s["scale"]
        w_all.append(w.detach())
        i_all.append(idx.to(torch.int32))
        if s["train"]:
            d_all.append(torch.autograd.grad(w, l, s["dw"][a:a + 512].double())[0])
    return [torch.cat(v) for v in ([w_all, i_all, d_all] if s["train"] else [w_all, i_all])]


def _exact_experts(s):
    import numpy as np
    T, k, H, E = s["T"], s["k"], s["H"], s["E"]
    e = s["experts"].cpu().numpy().reshape(-1).astype(np.int64)
    e[e < 0] = E
    order = np.lexsort((np.arange(e.size), e))
    slots = np.empty(e.size, dtype=np.int64)
    slots[order] = np.arange(e.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(e, minlength=E + 1)[:E])])
    live = int(offsets[E])
    order_t = torch.from_numpy(order).to(device)
    slots_t = torch.from_numpy(slots).to(device).view(T, k)
    x, y, w = (s[i].detach() for i in ("x", "y", "w"))
    xs = torch.zeros((T * k, H), dtype=x.dtype, device=device)
    xs[:live] = x[order_t[:live] // k]
    out = torch.zeros((T, H), dtype=torch.float64, device=device)
    for j in range(k):
        at = slots_t[:, j]
        ok = at < live
        out[ok] += w[ok, j, None].double() * y[at[ok]].double()
    i32 = lambda v: torch.from_numpy(v.astype(np.int32)).to(device)  # noqa: E731
    got = [i32(offsets), i32(slots).view(T, k), i32(order), xs, out]
    if s["train"]:
        dx = torch.zeros((T, H), dtype=torch.float64, device=device)
        dw = torch.zeros((T, k), dtype=torch.float64, device=device)
        dy = torch.zeros((T * k, H), dtype=torch.float64, device=device)
        g = s["dout"].double()
        for j in range(k):
            at = slots_t[:, j]
            ok = at < live
            dx[ok] += s["dxs"][at[ok]].double()
            dw[ok, j] = torch.einsum("th,th->t", g[ok], y[at[ok]].double())
            dy[at[ok]] = w[ok, j, None].double() * g[ok]
        got += [dx, dy, dw]
    return got


def _exact_attend(s):
    B, Hkv, G, Sq, D = (s[i] for i in ("B", "Hkv", "G", "Sq", "D"))
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=device)
    score = s["score"].double()
    for b, n in enumerate(s["lengths"].tolist()):
        sees = torch.arange(n, device=device)[None, :] <= (n - Sq + torch.arange(Sq, device=device))[:, None]
        some = sees.any(1)
        for h in range(Hkv):
            kd, vd = s["kc"][b, h, :n].double(), s["vc"][b, h, :n].double()
            for g in range(G):
                a = torch.einsum("id,nd->in", s["q"][b, :, h * G + g].double(), kd) / math.sqrt(D)
                p = torch.softmax(a.masked_fill(~sees, -math.inf), 1)
                p = torch.where(some[:, None], p, 0.0)
                out[b, :, h * G + g] = torch.einsum("in,nd->id", p, vd)
                score[b, h, :n] += p.sum(0)
    return [out, score]


def _exact_evict(s):
    import numpy as np
    B, Hkv, budget = s["B"], s["Hkv"], s["budget"]
    score, lengths = s["score"].cpu().numpy().astype(np.float64), s["lengths"].cpu().numpy()
    pos = np.full((B, Hkv, budget), -1, dtype=np.int64)
    for b in range(B):
        n = int(lengths[b])
        held = np.zeros(n, dtype=bool)
        held[:s["first"]] = True
        held[max(0, n - s["last"]):] = True
        for h in range(Hkv):
            if n <= budget:
                pos[b, h, :n] = np.arange(n)
                continue
            free = np.flatnonzero(~held)
            take = budget - int(held.sum())
            best = free[np.lexsort((free, -score[b, h, free]))[:take]]
            pos[b, h] = np.sort(np.concatenate([np.flatnonzero(held), best]))
    p = torch.from_numpy(pos).to(device)
    at = p.clamp(min=0)
    take = lambda c: (c[torch.arange(B, device=device)[:, None, None], torch.arange(Hkv, device=device)[None, :, None], at]  # noqa: E731
                      * (p >= 0)[..., None].to(c.dtype))
    left = torch.from_numpy(np.minimum(lengths, budget).astype(np.int32)).to(device)
    return [take(s["kc"]), take(s["vc"]), take(s["score"][..., None])[..., 0].double(), p.to(torch.int32), left]


def exact(case, seed):
    s = prepare(case, seed)
    return globals()["_exact_" + case["op"]](s)
