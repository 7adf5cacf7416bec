"""Measured cases of the operators around the MoE experts' products: routing
tokens to experts, moving them into expert order and back, and the global
gradient norm with clipping.

``run`` computes a case in plain torch operations, or, with ``own`` set,
through this repository's entry points.  Sizes: the MoE workload (16384 tokens,
top 8 of 64 experts, hidden 4096), the linear stack's weights (7168 and
18432), single tokens, and ragged sizes in between.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

NEG = -math.inf


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token of a decoding step, router logits in FP32: launch latency
        dict(name="route_one_token", op="route", tokens=1, experts=64, top_k=8, dtype="float32",
             score="softmax", bias=False, groups=1, top_groups=1, renorm=True, scale=1.0, pad=0.0),
        # the MoE workload's training batch
        dict(name="route_layer", op="route", tokens=16384, experts=64, top_k=8, dtype="bfloat16",
             score="softmax", bias=False, groups=1, top_groups=1, renorm=True, scale=1.0, pad=0.0),
        # a large batch with sigmoid scores, a balance bias and expert groups; one
        # token in 20 is padding, whose logits are all masked
        dict(name="route_groups", op="route", tokens=65536, experts=256, top_k=8, dtype="float32",
             score="sigmoid", bias=True, groups=8, top_groups=4, renorm=True, scale=2.5, pad=0.05),
        # training with plain softmax weights: a dense gradient
        dict(name="route_backward_softmax", op="route_backward", tokens=16384, experts=64, top_k=8,
             dtype="float32", score="softmax", renorm=False, scale=1.0),
        # a ragged batch, odd number of experts, BF16 logits
        dict(name="route_backward_sigmoid", op="route_backward", tokens=30011, experts=250, top_k=6,
             dtype="bfloat16", score="sigmoid", renorm=True, scale=2.5),
        # the MoE workload's tokens as the gate_up product reads them
        dict(name="dispatch_quant_layer", op="dispatch_quant", tokens=16384, experts=64, top_k=8,
             hidden=4096, elem="e4m3", drop=0.0),
        # a small ragged batch with dropped choices, in BF16
        dict(name="dispatch_ragged", op="dispatch", tokens=1021, experts=60, top_k=3, hidden=1000,
             drop=0.1),
        # the MoE workload's down-projection result back to the tokens
        dict(name="combine_layer", op="combine", tokens=16384, experts=64, top_k=8, hidden=4096,
             residual=True, weighted=True, drop=0.0),
        # one token of a decoding step
        dict(name="combine_one_token", op="combine", tokens=1, experts=64, top_k=8, hidden=7168,
             residual=False, weighted=True, drop=0.0),
        # the MoE workload's backward pass
        dict(name="combine_backward_layer", op="combine_backward", tokens=16384, experts=64,
             top_k=8, hidden=4096, drop=0.0),
        # the norms, biases and router of a small model: many short odd tensors
        dict(name="grad_norm_small", op="grad_norm", matrices=2, rows=61, cols=257, vectors=11,
             clip=False, ratio=0.1),
        # the linear stack's weight gradients in BF16 with its FP32 vectors, clipped
        dict(name="grad_clip_stack", op="grad_norm", matrices=8, rows=18432, cols=7168, vectors=40,
             clip=True, ratio=0.1),
    ]


def _log(rng, lo, hi, unit=1):
    """A multiple of unit, spread over the logarithm; off the round sizes,
    which the listed cases stand for."""
    n = unit * max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n - unit if n % 1024 == 0 and n > unit else n


def draw(rng):
    op = rng.choice(["route", "route_backward", "dispatch_quant", "dispatch", "combine",
                     "combine_backward", "grad_norm"])
    if op == "grad_norm":
        cols = _log(rng, 16, 7168)
        return dict(op=op, matrices=rng.randint(1, 8), rows=_log(rng, 16, 18432), cols=cols,
                    vectors=rng.randint(0, 40), clip=rng.random() < 0.6,
                    ratio=rng.choice([0.01, 0.1, 0.5, 2.0]))
    experts = rng.choice([8, 16, 32, 60, 64, 96, 128, 160, 250, 256, 384, 512, rng.randint(5, 512)])
    top_k = rng.randint(1, min(12, experts))
    if op in ("route", "route_backward"):
        tokens = _log(rng, 1, max(1, 65536 * 256 // max(experts, 256)))
        dtype = rng.choice(["float32", "bfloat16"])
        score = rng.choice(["softmax", "sigmoid"])
        renorm, scale = rng.random() < 0.6, rng.choice([1.0, 2.5])
        if op == "route_backward":
            # a single renormalised weight is constant: its gradient is 0
            return dict(op=op, tokens=tokens, experts=experts, top_k=top_k, dtype=dtype,
                        score=score, renorm=renorm and top_k > 1, scale=scale)
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if experts % g == 0])
        top_groups = rng.randint((groups + 1) // 2, groups)
        top_k = min(top_k, top_groups * (experts // groups))
        return dict(op=op, tokens=tokens, experts=experts, top_k=top_k, dtype=dtype, score=score,
                    bias=rng.random() < 0.5, groups=groups, top_groups=top_groups, renorm=renorm,
                    scale=scale, pad=rng.choice([0.0, 0.0, 0.1]))
    hidden = _log(rng, 4, 256, 32) if op == "dispatch_quant" or rng.random() < 0.6 \
        else _log(rng, 100, 8192)
    tokens = _log(rng, 1, max(1, min(16384, 16384 * 8 * 4096 // (top_k * hidden))))
    c = dict(op=op, tokens=tokens, experts=experts, top_k=top_k, hidden=hidden,
             drop=rng.choice([0.0, 0.0, 0.05, 0.3]) if tokens >= 16 else 0.0)
    if op == "dispatch_quant":
        c["elem"] = rng.choice(["e4m3", "e5m2"])
    if op == "combine":
        c["residual"], c["weighted"] = rng.random() < 0.5, rng.random() < 0.7
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _logits(tokens, experts, dtype, g, pad=0.0):
    """Router logits: some experts are preferred by all tokens; padding
    tokens have every expert masked."""
    x = 1.3 * _randn((tokens, experts), g) + 0.6 * _randn((1, experts), g)
    if pad:
        x[torch.rand((tokens,), generator=g, device="cuda") < pad] = NEG
    return x.to(getattr(torch, dtype))


def _layout(experts, n_experts):
    """Expert-ordered rows of the choices experts [T, k] (-1: none): the
    offsets [E + 1] and each choice's row (-1: none)."""
    flat = experts.flatten().long()
    key = torch.where(flat < 0, n_experts, flat)
    order = torch.sort(key, stable=True).indices
    slots = torch.empty_like(key)
    slots[order] = torch.arange(key.numel(), device=key.device)
    slots = torch.where(flat < 0, -1, slots).to(torch.int32).view(experts.shape)
    counts = torch.zeros(n_experts + 1, dtype=torch.int64, device=key.device)
    counts.scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([torch.zeros_like(counts[:1]), torch.cumsum(counts[:n_experts], 0)])
    return offsets, slots


def _routing(case, g):
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    score = _randn((T, E), g) + 0.6 * _randn((1, E), g)
    experts = torch.sort(score, dim=1, descending=True).indices[:, :k].to(torch.int32)
    if case["drop"]:
        experts[torch.rand((T, k), generator=g, device="cuda") < case["drop"]] = -1
    weights = torch.rand((T, k), generator=g, device="cuda") + 0.1
    weights = weights / weights.sum(1, keepdim=True)
    weights = torch.where(experts < 0, torch.zeros_like(weights), weights)
    offsets, slots = _layout(experts, E)
    return dict(weights=weights, experts=experts.contiguous(), offsets=offsets, slots=slots)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op == "route":
        s["logits"] = _logits(case["tokens"], case["experts"], case["dtype"], g, case["pad"])
        s["bias"] = 0.05 * _randn((case["experts"],), g) if case["bias"] else None
    elif op == "route_backward":
        s["logits"] = _logits(case["tokens"], case["experts"], case["dtype"], g)
        s["experts"] = torch.sort(s["logits"].float(), dim=1, descending=True,
                                  stable=True).indices[:, :case["top_k"]].to(torch.int32)
        s["experts"] = s["experts"].contiguous()
        s["dweights"] = _randn((case["tokens"], case["top_k"]), g)
    elif op == "grad_norm":
        mats = [(0.01 * _randn((case["rows"], case["cols"]), g)).to(torch.bfloat16)
                for _ in range(case["matrices"])]
        vecs = [0.01 * _randn((case["cols"] + 3 * i,), g) for i in range(case["vectors"])]
        s["tensors"] = mats + vecs
        n = sum(t.numel() for t in s["tensors"])
        s["max_norm"] = case["ratio"] * 0.01 * math.sqrt(n)
    else:
        T, k, H = case["tokens"], case["top_k"], case["hidden"]
        s["routing"] = _routing(case, g)
        if op in ("dispatch", "dispatch_quant"):
            s["x"] = _randn((T, H), g).to(torch.bfloat16)
        else:
            s["y"] = _randn((T * k, H), g).to(torch.bfloat16)
        if op == "combine":
            s["residual"] = _randn((T, H), g).to(torch.bfloat16) if case["residual"] else None
        if op == "combine_backward":
            s["dout"] = (0.01 * _randn((T, H), g)).to(torch.bfloat16)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    import mxfp8_microscaled_precision_amd as mx
    c = s["case"]
    op = c["op"]
    if op == "route":
        r = mx.route(s["logits"], c["top_k"], c["score"], s["bias"], n_groups=c["groups"],
                     top_groups=c["top_groups"], renormalize=c["renorm"], scale=c["scale"])
        return dict(weights=r.weights, experts=r.experts, offsets=r.offsets, slots=r.slots)
    if op == "route_backward":
        return mx.route_backward(s["dweights"], s["logits"], s["experts"], c["score"],
                                 renormalize=c["renorm"], scale=c["scale"])
    if op == "grad_norm":
        if c["clip"]:
            return mx.grad_clip(s["tensors"], s["max_norm"]), s["tensors"]
        return mx.grad_norm(s["tensors"])
    r = mx.Routing(**s["routing"])
    if op == "dispatch":
        return mx.dispatch(s["x"], r)
    if op == "dispatch_quant":
        q, sc = mx.dispatch_quant(s["x"], r, c["elem"])
        return q.view(_ELEM[c["elem"]][0]), sc
    if op == "combine":
        return mx.combine(s["y"], r, residual=s["residual"], weighted=c["weighted"])
    return mx.combine_backward(s["dout"], s["y"], r)


def _plain_scores(x, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    m = x.amax(1, keepdim=True)
    p = torch.exp(x - torch.where(m == NEG, torch.zeros_like(m), m))
    tot = p.sum(1, keepdim=True)
    return p / torch.where(tot > 0, tot, torch.ones_like(tot))


def _plain_route(s):
    # in 64 bits: the choice turns on scores that lie next to each other
    c, x = s["case"], s["logits"].double()
    T, E = x.shape
    scores = _plain_scores(x, c["score"])
    sel = scores if s["bias"] is None else scores + s["bias"].double()
    sel = torch.where(x == NEG, NEG, sel)
    if c["groups"] > 1:
        by = sel.view(T, c["groups"], -1)
        best = torch.sort(by, dim=2, descending=True).values[:, :, :2]
        val = torch.where(best[:, :, -1] == NEG, best[:, :, 0], best.sum(2)) \
            if best.shape[2] > 1 else best[:, :, 0]
        keep = torch.sort(val, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        on = torch.zeros((T, c["groups"]), dtype=torch.bool, device=x.device).scatter_(1, keep, True)
        sel = torch.where(on[:, :, None], by, NEG).view(T, E)
    v, idx = torch.sort(sel, dim=1, descending=True, stable=True)
    v, idx = v[:, :c["top_k"]], idx[:, :c["top_k"]]
    u = torch.where(v == NEG, 0.0, scores.gather(1, idx))
    if c["renorm"]:
        tot = u.sum(1, keepdim=True)
        u = u / torch.where(tot > 0, tot, torch.ones_like(tot))
    experts = torch.where(v == NEG, -1, idx).to(torch.int32)
    offsets, slots = _layout(experts, E)
    return dict(weights=(c["scale"] * u).float(), experts=experts, offsets=offsets, slots=slots)


def _plain_route_backward(s):
    c, x = s["case"], s["logits"].float()
    scores = _plain_scores(x, c["score"])
    idx = s["experts"].long()
    u = scores.gather(1, idx)
    g = c["scale"] * s["dweights"]
    if c["renorm"]:
        tot = u.sum(1, keepdim=True)
        g = (g - (g * u).sum(1, keepdim=True) / tot) / tot
    ds = torch.zeros_like(scores).scatter_(1, idx, g)
    if c["score"] == "sigmoid":
        dx = ds * scores * (1.0 - scores)
    else:
        dx = scores * (ds - (ds * scores).sum(1, keepdim=True))
    return dx.to(s["logits"].dtype)


# payload type, largest finite value, mantissa bits, smallest normal exponent
_ELEM = {"e4m3": (torch.float8_e4m3fn, 448.0, 3, -6), "e5m2": (torch.float8_e5m2, 57344.0, 2, -14)}


def _spread(rows, slots):
    """out[slot] = rows[t] for every choice; rows that no choice takes are 0."""
    T, k = slots.shape
    out = torch.zeros((T * k + 1,) + rows.shape[1:], dtype=rows.dtype, device=rows.device)
    to = torch.where(slots < 0, T * k, slots).long().flatten()
    out[to] = rows[:, None].expand(T, k, *rows.shape[1:]).reshape(T * k, *rows.shape[1:])
    out[T * k] = 0
    return out[:T * k]


def _plain_dispatch(s):
    return _spread(s["x"], s["routing"]["slots"])


def _plain_dispatch_quant(s):
    kind, big = _ELEM[s["case"]["elem"]][:2]
    x = s["x"].float()
    blocks = x.view(x.shape[0], -1, 32)
    amax = blocks.abs().amax(2)
    # the smallest e with amax <= big * 2^e
    mant, e = torch.frexp(amax / big)
    e = torch.where(mant == 0.5, e - 1, e)
    e = torch.where(amax == 0, -127, e).clamp(-127, 126).to(torch.int32)
    inv = ((127 - e) << 23).view(torch.float32)                     # 2^-e
    q = (blocks * inv[:, :, None]).clamp(-big, big).to(kind).view(torch.uint8)
    slots = s["routing"]["slots"]
    q = _spread(q.view(x.shape), slots)
    return q.view(kind), _spread((e + 127).to(torch.uint8), slots)


def _plain_combine(s):
    r = s["routing"]
    T, k = r["slots"].shape
    rows = s["y"][r["slots"].clamp(min=0).long().flatten()].float().view(T, k, -1)
    w = r["weights"] if s["case"]["weighted"] else torch.ones_like(r["weights"])
    w = torch.where(r["slots"] < 0, torch.zeros_like(w), w)
    out = (rows * w[:, :, None]).sum(1)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return out.to(torch.bfloat16)


def _plain_combine_backward(s):
    r = s["routing"]
    T, k = r["slots"].shape
    d = s["dout"].float()
    dropped = r["slots"] < 0
    rows = s["y"][r["slots"].clamp(min=0).long().flatten()].float().view(T, k, -1)
    dw = torch.where(dropped, 0.0, (rows * d[:, None]).sum(2))
    part = (r["weights"][:, :, None] * d[:, None]).to(torch.bfloat16)
    dy = torch.zeros((T * k + 1, d.shape[1]), dtype=torch.bfloat16, device=d.device)
    dy[torch.where(dropped, T * k, r["slots"]).long().flatten()] = part.view(T * k, -1)
    dy[T * k] = 0
    return dy[:T * k], dw


def _plain_grad_norm(s):
    # squares in 32 bits, their long sums in 64
    parts = [t.float().square().sum(dtype=torch.float64) for t in s["tensors"]]
    norm = torch.stack(parts).sum().sqrt().float()
    if not s["case"]["clip"]:
        return norm
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    return norm, [t.copy_(t.float() * coef) for t in s["tensors"]]


_PLAIN = dict(route=_plain_route, route_backward=_plain_route_backward, dispatch=_plain_dispatch,
              dispatch_quant=_plain_dispatch_quant, combine=_plain_combine,
              combine_backward=_plain_combine_backward, grad_norm=_plain_grad_norm)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "grad_norm":
        n16 = case["matrices"] * case["rows"] * case["cols"]
        n32 = sum(case["cols"] + 3 * i for i in range(case["vectors"]))
        each = 2 if case["clip"] else 1                 # read, and written where clipped
        return dict(bytes=each * (2 * n16 + 4 * n32) + 4, flops=(2 + case["clip"]) * (n16 + n32))
    T, E, k = case["tokens"], case["experts"], case["top_k"]
    P = T * k
    if op in ("route", "route_backward"):
        size = 2 if case["dtype"] == "bfloat16" else 4
        if op == "route":
            return dict(bytes=T * E * size + 12 * P + 8 * (E + 1) + 4 * E * case["bias"],
                        flops=8 * T * E)
        return dict(bytes=2 * T * E * size + 8 * P, flops=8 * T * E)
    H = case["hidden"]
    if op == "dispatch":
        return dict(bytes=2 * T * H + 2 * P * H + 4 * P + 8, flops=0)
    if op == "dispatch_quant":
        return dict(bytes=2 * T * H + P * H + P * H // 32 + 4 * P + 8, flops=2 * T * H)
    if op == "combine":
        return dict(bytes=2 * P * H + 2 * T * H * (1 + case["residual"]) + 4 * P * (1 + case["weighted"]),
                    flops=2 * P * H)
    return dict(bytes=2 * T * H + 4 * P * H + 12 * P + 8, flops=3 * P * H)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return _EXACT[case["op"]](case, s)


def _exact_route(c, s):
    x = s["logits"].double().cpu().numpy()
    T, E = x.shape
    k, n = c["top_k"], c["groups"]
    with np.errstate(invalid="ignore", over="ignore"):
        if c["score"] == "softmax":
            z = x - x.max(1, keepdims=True)
            z = np.exp(z)
            score = z / z.sum(1, keepdims=True)
        else:
            score = np.reciprocal(1 + np.exp(-x))
    v = score.copy()
    if s["bias"] is not None:
        v += s["bias"].double().cpu().numpy()
    v[np.isneginf(x)] = NEG
    if n > 1:
        by = np.sort(v.reshape(T, n, E // n), axis=2)[:, :, ::-1]
        val = by[:, :, 0].copy()
        if E // n > 1:
            two = by[:, :, 1]
            val[~np.isneginf(two)] += two[~np.isneginf(two)]
        rank = np.argsort(np.argsort(-val, axis=1, kind="stable"), axis=1, kind="stable")
        v[np.repeat(rank >= c["top_groups"], E // n, axis=1)] = NEG
    at = np.argsort(-v, axis=1, kind="stable")[:, :k]
    none = np.isneginf(np.take_along_axis(v, at, 1))
    w = np.where(none, 0, np.take_along_axis(score, at, 1))
    if c["renorm"]:
        tot = w.sum(1, keepdims=True)
        w = np.divide(w, tot, out=np.zeros_like(w), where=tot > 0)
    experts = np.where(none, -1, at).astype(np.int32)
    flat = experts.ravel()
    kept = np.flatnonzero(flat >= 0)
    kept = kept[np.argsort(flat[kept], kind="stable")]
    slots = np.full(flat.size, -1, np.int32)
    slots[kept] = np.arange(kept.size, dtype=np.int32)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[flat >= 0], minlength=E))])
    return dict(weights=c["scale"] * w, experts=experts, offsets=offsets.astype(np.int64),
                slots=slots.reshape(T, k))


def _exact_route_backward(c, s):
    # the weights' derivative, choice by choice, from the chosen scores
    x, e = s["logits"].double(), s["experts"].long()
    g, scale = s["dweights"].double(), c["scale"]
    if c["score"] == "softmax":
        p = torch.exp(x - torch.logsumexp(x, 1, keepdim=True))
    else:
        p = torch.sigmoid(x)
    u = p.gather(1, e)
    if c["renorm"]:
        a = u / u.sum(1, keepdim=True)
        d = scale * a * (g - (g * a).sum(1, keepdim=True))
        if c["score"] == "sigmoid":
            d = d * (1 - u)
        return torch.zeros_like(x).scatter_(1, e, d)
    if c["score"] == "sigmoid":
        return torch.zeros_like(x).scatter_(1, e, scale * g * u * (1 - u))
    d = -scale * p * (g * u).sum(1, keepdim=True)
    return d.scatter_add_(1, e, scale * g * u)


def _exact_rows(slots, value):
    """out [T k, H] in 64 bits: value(j) [T, H] at the rows of choice j."""
    T, k = slots.shape
    out = None
    for j in range(k):
        v = value(j)
        if out is None:
            out = torch.zeros((T * k,) + v.shape[1:], dtype=v.dtype, device=v.device)
        on = slots[:, j] >= 0
        out[slots[on, j].long()] = v[on]
    return out


def _exact_dispatch(c, s):
    x = s["x"].double()
    return _exact_rows(s["routing"]["slots"], lambda j: x)


def _pow2(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_dispatch_quant(c, s):
    _, big, bits, low = _ELEM[c["elem"]]
    x = s["x"].double()
    b = x.view(x.shape[0], -1, 32)
    amax = b.abs().amax(2)
    e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -133) / big))
    e = torch.where(amax > big * _pow2(e), e + 1, e)           # log2 may round across a power
    e = torch.where(amax <= big * _pow2(e - 1), e - 1, e).clamp(-127, 127)
    v = b / _pow2(e)[:, :, None]
    step = _pow2(torch.floor(torch.log2(v.abs().clamp(min=1e-300))).clamp(min=low) - bits)
    v = (torch.round(v / step) * step).view(x.shape)                # ties to even
    slots = s["routing"]["slots"]
    q = _exact_rows(slots, lambda j: v)
    return q, _exact_rows(slots, lambda j: e + 127).to(torch.uint8)


def _exact_combine(c, s):
    r = s["routing"]
    out = torch.zeros((c["tokens"], c["hidden"]), dtype=torch.float64, device="cuda")
    if s["residual"] is not None:
        out += s["residual"]
    for j in range(c["top_k"]):
        on = (r["slots"][:, j] >= 0).nonzero().flatten()
        w = r["weights"][on, j].double() if c["weighted"] else torch.ones_like(on).double()
        out[on] += w[:, None] * s["y"][r["slots"][on, j].long()].double()
    return out


def _exact_combine_backward(c, s):
    r, d = s["routing"], s["dout"].double()
    dw = torch.zeros(r["weights"].shape, dtype=torch.float64, device="cuda")
    for j in range(c["top_k"]):
        on = (r["slots"][:, j] >= 0).nonzero().flatten()
        dw[on, j] = (d[on] * s["y"][r["slots"][on, j].long()].double()).sum(1)
    dy = _exact_rows(r["slots"], lambda j: r["weights"][:, j:j + 1].double() * d)
    return dy, dw


def _exact_grad_norm(c, s):
    norm = math.sqrt(math.fsum(float((t.double() ** 2).sum()) for t in s["tensors"]))
    if not c["clip"]:
        return norm
    coef = min(1.0, s["max_norm"] / (norm + 1e-6))
    return norm, [t.double() * coef for t in s["tensors"]]


_EXACT = dict(route=_exact_route, route_backward=_exact_route_backward, dispatch=_exact_dispatch,
              dispatch_quant=_exact_dispatch_quant, combine=_exact_combine,
              combine_backward=_exact_combine_backward, grad_norm=_exact_grad_norm)
