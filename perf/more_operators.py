"""Measured cases of the operators around 4-bit weights and 8-bit activation
checkpoints: microscaled E2M1 quantisation, the dense and grouped products
with E2M1 weights, the SwiGLU with its quantised result and its gate/up
checkpoint, the gradient from that checkpoint, and the column blocks of a
weight gradient's operand from the row blocks kept by the forward pass.

``run`` computes a case in plain torch operations, or, with ``own`` set,
through this repository's entry points.  Sizes: the linear stack (7168 and
18432, 32768 tokens), the MoE workload (131072 routed rows, 64 experts, hidden
4096, expert width 2048), single tokens, and ragged sizes in between.
"""
from __future__ import annotations

import math

import torch

own = False

# largest finite value, mantissa bits, exponent of the smallest normal value
FORMAT = {"e4m3": (448.0, 3, -6), "e5m2": (57344.0, 2, -14), "e2m1": (6.0, 1, 0)}
FLOAT8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # a layer's weight, quantised for the forward and the backward product
        # after an optimiser step, and restored (quantisation-aware training)
        dict(name="quant4_weight", op="quant4", rows=18432, cols=7168, mode="dual"),
        # a ragged batch of activations in rows
        dict(name="quant4_ragged", op="quant4", rows=1021, cols=4128, mode="row"),
        # one token of a decoding step through a layer with 4-bit weights
        dict(name="gemm4_one_token", op="gemm4", M=1, N=18432, K=7168, a_elem="e4m3"),
        # a short ragged batch, E5M2 gradients against the 4-bit weight
        dict(name="gemm4_ragged", op="gemm4", M=1021, N=4130, K=2080, a_elem="e5m2"),
        # the linear stack's training batch, both operands in 4 bits
        dict(name="gemm4_layer", op="gemm4", M=32768, N=18432, K=7168, a_elem="e2m1"),
        # 16 sequences' tokens of a decoding step, top 8 of 64 experts
        dict(name="grouped4_decode", op="grouped4", T=128, G=64, N=4096, K=4096, a_elem="e4m3",
             skew=0.5),
        # the MoE workload's gate_up product
        dict(name="grouped4_layer", op="grouped4", T=131072, G=64, N=4096, K=4096, a_elem="e4m3",
             skew=0.5),
        # between the MoE workload's two products, with the checkpoint
        dict(name="swiglu_layer", op="swiglu", T=131072, F=2048, elem="e4m3", checkpoint=True),
        # one token of a decoding step, dense layer, no checkpoint
        dict(name="swiglu_one_token", op="swiglu", T=1, F=18432, elem="e4m3", checkpoint=False),
        # the MoE workload's backward pass between the two products
        dict(name="swiglu_backward_layer", op="swiglu_backward", T=131072, F=2048, elem="bf16"),
        # the MoE workload's gate_up input, in column blocks for its weight gradient
        dict(name="requant_grouped_layer", op="requant", T=131072, C=4096, G=64, elem="e4m3",
             out_elem="e4m3", skew=0.5),
        # a small dense layer's E5M2 gradient
        dict(name="requant_small", op="requant", T=1056, C=2080, G=0, elem="e5m2",
             out_elem="e5m2", skew=0.0),
    ]


def _log(rng, lo, hi, unit=1):
    """A multiple of unit, spread over the logarithm; off the round sizes,
    which the listed cases stand for."""
    n = unit * max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))
    return n - unit if n % 1024 == 0 and n > unit else n


def draw(rng):
    op = rng.choice(["quant4", "gemm4", "gemm4", "grouped4", "swiglu", "swiglu_backward", "requant"])
    if op == "quant4":
        mode = rng.choice(["row", "col", "dual"])
        cols = _log(rng, 1, 576, 32)
        rows = _log(rng, 1, 18432) if mode == "row" else _log(rng, 1, 224, 32)
        return dict(op=op, rows=rows, cols=cols, mode=mode)
    if op == "gemm4":
        K = _log(rng, 1, 576, 32)
        N = _log(rng, 1, 18432)
        M = _log(rng, 1, 32768 * 18432 * 7168 // (18432 * 18432) if K > 7168 else 32768)
        return dict(op=op, M=M, N=N, K=K, a_elem=rng.choice(["e4m3", "e5m2", "e2m1"]))
    if op == "grouped4":
        return dict(op=op, T=_log(rng, 1, 32768), G=rng.choice([1, 8, 16, 60, 64, rng.randint(2, 64)]),
                    N=_log(rng, 32, 4096), K=_log(rng, 1, 128, 32),
                    a_elem=rng.choice(["e4m3", "e5m2", "e2m1"]), skew=rng.choice([0.0, 0.5, 1.0]))
    if op in ("swiglu", "swiglu_backward"):
        F = _log(rng, 1, 576, 32)
        c = dict(op=op, T=_log(rng, 1, min(131072, 131072 * 2048 // F)), F=F)
        if op == "swiglu":
            return dict(c, elem="e4m3", checkpoint=rng.random() < 0.7)
        return dict(c, elem=rng.choice(["bf16", "e4m3"]))
    G = rng.choice([0, 0, 1, 8, 60, 64, rng.randint(2, 64)])
    C = _log(rng, 1, 576, 32)
    T = _log(rng, 1, min(4096, 131072 * 4096 // (32 * C)), 32) - (rng.randint(0, 31) if G else 0)
    return dict(op=op, T=T, C=C, G=G, elem=rng.choice(["e4m3", "e5m2"]),
                out_elem=rng.choice(["e4m3", "e5m2"]), skew=rng.choice([0.0, 0.5, 1.0]) if G else 0.0)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _operand(rows, cols, std, elem, g):
    """A quantised normal matrix as a user holds it: payload and scales, with
    row magnitudes that differ."""
    x = _randn((rows, cols), g) * std * torch.exp(0.3 * _randn((rows, 1), g))
    v, s = _plain_quant(x.to(torch.bfloat16).float(), elem)
    return _payload(v, elem), s


def _offsets(T, G, skew, g):
    """T rows over G groups, whose shares differ by exp(skew n)."""
    share = torch.exp(skew * _randn((G,), g))
    edge = torch.sort(torch.multinomial(share, T, replacement=True, generator=g)).values
    return torch.searchsorted(edge, torch.arange(G + 1, device="cuda"))


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op == "quant4":
        s["x"] = (0.02 * _randn((case["rows"], case["cols"]), g)).to(torch.bfloat16)
    elif op == "gemm4":
        s["a"], s["sa"] = _operand(case["M"], case["K"], 1.0, case["a_elem"], g)
        s["b"], s["sb"] = _operand(case["N"], case["K"], 0.02, "e2m1", g)
    elif op == "grouped4":
        s["a"], s["sa"] = _operand(case["T"], case["K"], 1.0, case["a_elem"], g)
        experts = [_operand(case["N"], case["K"], 0.02, "e2m1", g) for _ in range(case["G"])]
        s["b"] = torch.stack([e[0] for e in experts])
        s["sb"] = torch.stack([e[1] for e in experts])
        s["offsets"] = _offsets(case["T"], case["G"], case["skew"], g)
        # rows of the largest group, which the plain form pads to
        s["most"] = max(1, int(torch.diff(s["offsets"]).max()))
    elif op == "swiglu":
        s["gate_up"] = (1.2 * _randn((case["T"], 2 * case["F"]), g)).to(torch.bfloat16)
    elif op == "swiglu_backward":
        s["q"], s["s"] = _operand(case["T"], 2 * case["F"], 1.2, "e4m3", g)
        s["dh"] = (0.01 * _randn((case["T"], case["F"]), g)).to(torch.bfloat16)
    else:
        s["q"], s["s"] = _operand(case["T"], case["C"], 1.0, case["elem"], g)
        if case["G"]:
            s["offsets"] = _offsets(case["T"], case["G"], case["skew"], g)
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
    if op == "quant4":
        out = mx.quant4(s["x"], c["mode"])
        return [(mx.dequant(q, sc, "e2m1"), sc) for q, sc in zip(out[::2], out[1::2])]
    if op == "gemm4":
        return mx.gemm4(s["a"], s["sa"], s["b"], s["sb"], c["a_elem"])
    if op == "grouped4":
        return mx.grouped_gemm4(s["offsets"], s["a"], s["sa"], s["b"], s["sb"], c["a_elem"])
    if op == "swiglu":
        q, sc, ckpt = mx.swiglu_quant(s["gate_up"], c["elem"], checkpoint=c["checkpoint"])
        out = [q.view(FLOAT8[c["elem"]]), sc.view(torch.float8_e8m0fnu)]
        return out + ([ckpt[0].view(FLOAT8["e4m3"]), ckpt[1]] if c["checkpoint"] else [])
    if op == "swiglu_backward":
        if c["elem"] == "bf16":
            return mx.swiglu_backward(s["dh"], s["q"], s["s"])
        q, sc = mx.swiglu_backward_quant(s["dh"], s["q"], s["s"], c["elem"])
        return q.view(FLOAT8[c["elem"]]), sc.view(torch.float8_e8m0fnu)
    if c["G"]:
        q, sc = mx.requant_grouped_col(s["q"], s["s"], s["offsets"], c["elem"], c["out_elem"])
    else:
        q, sc = mx.requant_col(s["q"], s["s"], c["elem"], c["out_elem"])
    return q.view(FLOAT8[c["out_elem"]]), sc


def _pow2(e):
    """2^e in FP32 for integers e in [-126, 127]."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _plain_quant(x, elem):
    """Blocks of 32 along the last axis of x FP32: the values that the codes
    stand for, before the scale, and the scale bytes."""
    big, bits, low = FORMAT[elem]
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1)
    # the smallest e with amax <= big * 2^e
    mant, e = torch.frexp(amax / big)
    e = torch.where(mant == 0.5, e - 1, e)
    e = torch.where(amax == 0, -127, e).clamp(-127, 126).to(torch.int32)
    v = b * _pow2(-e)[..., None]
    if elem != "e2m1":
        v = v.clamp(-big, big).to(FLOAT8[elem])
    else:
        a = v.abs()
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        v = torch.copysign(torch.round(a / step) * step, v)         # ties to even
    return v.view(x.shape), (e + 127).to(torch.uint8)


def _payload(v, elem):
    """The stored bytes of code values."""
    if elem != "e2m1":
        return v.view(torch.uint8)
    a = v.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code + 8 * torch.signbit(v).to(torch.uint8)
    return code[..., ::2] | (code[..., 1::2] << 4)


def _plain_values(q, s, elem):
    """Payload and scales back to FP32 values."""
    if elem != "e2m1":
        v = q.view(FLOAT8[elem]).float()
    else:
        code = torch.stack([q & 15, q >> 4], -1).view(*q.shape[:-1], -1)
        m, e = (code & 1).float(), ((code >> 1) & 3).to(torch.int32)
        v = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * _pow2(e - 1))
        v = torch.where(code > 7, -v, v)
    scale = (s.to(torch.int32) << 23).view(torch.float32)       # byte 0: a block of zeros
    return (v.view(*s.shape, 32) * scale[..., None]).view(v.shape)


def _plain_quant4(s):
    x, out = s["x"].float(), []
    for t in {"row": [x], "col": [x.t()], "dual": [x, x.t()]}[s["case"]["mode"]]:
        v, sc = _plain_quant(t, "e2m1")
        scale = (sc.to(torch.int32) << 23).view(torch.float32)
        out.append(((v.view(*sc.shape, 32) * scale[..., None]).view(v.shape).to(torch.bfloat16), sc))
    return out


def _plain_gemm4(s):
    a = _plain_values(s["a"], s["sa"], s["case"]["a_elem"])
    return torch.matmul(a, _plain_values(s["b"], s["sb"], "e2m1").t()).to(torch.bfloat16)


def _plain_grouped4(s):
    a = _plain_values(s["a"], s["sa"], s["case"]["a_elem"])
    b = _plain_values(s["b"], s["sb"], "e2m1")
    off, T = s["offsets"], a.shape[0]
    # every group padded to the largest one's rows
    at = off[:-1, None] + torch.arange(s["most"], device=a.device)
    on = at < off[1:, None]
    y = torch.matmul(a[at.clamp(max=T - 1)], b.transpose(1, 2))
    out = torch.empty((T, b.shape[1]), dtype=torch.bfloat16, device=a.device)
    out[at[on]] = y[on].to(torch.bfloat16)
    return out


def _plain_swiglu(s):
    c, x = s["case"], s["gate_up"].float()
    gate, up = x[:, :c["F"]], x[:, c["F"]:]
    h = gate / (1.0 + torch.exp(-gate)) * up
    q, sc = _plain_quant(h.to(torch.bfloat16).float(), c["elem"])
    out = [q, sc.view(torch.float8_e8m0fnu)]
    return out + list(_plain_quant(x, "e4m3")) if c["checkpoint"] else out


def _plain_swiglu_backward(s):
    c = s["case"]
    x = _plain_values(s["q"], s["s"], "e4m3")
    gate, up, dh = x[:, :c["F"]], x[:, c["F"]:], s["dh"].float()
    sig = 1.0 / (1.0 + torch.exp(-gate))
    d = torch.cat([dh * up * sig * (1.0 + gate * (1.0 - sig)), dh * gate * sig], 1).to(torch.bfloat16)
    if c["elem"] == "bf16":
        return d
    q, sc = _plain_quant(d.float(), c["elem"])
    return q, sc.view(torch.float8_e8m0fnu)


def _columns(off, T):
    """Source row of each column of the grouped layout, -1 where none is:
    group g's rows start at column 128 (off[g] // 128 + g)."""
    G = off.numel() - 1
    first = 128 * (off[:-1] // 128 + torch.arange(G, device=off.device))
    col = torch.arange(128 * (T // 128 + G), device=off.device)
    g = torch.searchsorted(first, col, right=True) - 1
    row = off[:-1][g] + col - first[g]
    return torch.where(row < off[1:][g], row, -1)


def _plain_requant(s):
    c = s["case"]
    x = _plain_values(s["q"], s["s"], c["elem"])
    if c["G"]:
        row = _columns(s["offsets"], c["T"])
        x = torch.where((row < 0)[:, None], 0.0, x[row.clamp(min=0)])
    return _plain_quant(x.t().contiguous(), c["out_elem"])


_PLAIN = dict(quant4=_plain_quant4, gemm4=_plain_gemm4, grouped4=_plain_grouped4,
              swiglu=_plain_swiglu, swiglu_backward=_plain_swiglu_backward, requant=_plain_requant)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    size = {"e4m3": 1 + 1 / 32, "e5m2": 1 + 1 / 32, "e2m1": 0.5 + 1 / 32, "bf16": 2}
    if op == "quant4":
        # x in, each copy's payload and scales out and in again, its values out
        n = case["rows"] * case["cols"]
        copies = 2 if case["mode"] == "dual" else 1
        return dict(bytes=n * (2 + copies * (2 * size["e2m1"] + 2)), flops=n * copies * 3)
    if op == "gemm4":
        M, N, K = case["M"], case["N"], case["K"]
        return dict(bytes=M * K * size[case["a_elem"]] + N * K * size["e2m1"] + 2 * M * N,
                    flops=2 * M * N * K)
    if op == "grouped4":
        T, N, K = case["T"], case["N"], case["K"]
        weights = min(case["G"], T) * N * K                     # of the groups that have rows, at most
        return dict(bytes=T * K * size[case["a_elem"]] + weights * size["e2m1"] + 2 * T * N,
                    flops=2 * T * N * K)
    if op == "swiglu":
        n = case["T"] * case["F"]
        return dict(bytes=n * (4 + size[case["elem"]] + 2 * size["e4m3"] * case["checkpoint"]),
                    flops=n * 8)
    if op == "swiglu_backward":
        n = case["T"] * case["F"]
        return dict(bytes=n * (2 + 2 * size["e4m3"] + 2 * size[case["elem"]]), flops=n * 14)
    n = case["T"] * case["C"]
    return dict(bytes=n * (size[case["elem"]] + size[case["out_elem"]]), flops=n * 4)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    return _EXACT[case["op"]](case, prepare(case, seed))


def _two(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_scale(x, elem):
    """Scale exponents of blocks of 32 along the last axis of x FP64."""
    big = FORMAT[elem][0]
    amax = x.abs().reshape(*x.shape[:-1], -1, 32).amax(-1)
    e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -130) / big))
    e = torch.where(amax > big * _two(e), e + 1, e)             # log2 may round across a power
    return torch.where(amax <= big * _two(e - 1), e - 1, e).clamp(-127, 127)


def _exact_codes(x, elem):
    """(code values, scale bytes) of blocks of 32, rounded to the format's grid."""
    big, bits, low = FORMAT[elem]
    e = _exact_scale(x, elem)
    v = x.reshape(*e.shape, 32) / _two(e)[..., None]
    step = _two(torch.floor(torch.log2(v.abs().clamp(min=1e-300))).clamp(min=low) - bits)
    return (torch.round(v / step) * step).reshape(x.shape), (e + 127).to(torch.uint8)


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _exact_values(q, s, elem):
    if elem == "e2m1":
        table = torch.tensor(_E2M1, dtype=torch.float64, device=q.device)
        v = torch.stack([table[(q & 15).long()], table[(q >> 4).long()]], -1).flatten(-2)
    else:
        v = q.view(FLOAT8[elem]).double()
    return (v.view(*s.shape, 32) * _two(s.int() - 127)[..., None]).view(v.shape)


def _exact_quant4(c, s):
    x, out = s["x"].double(), []
    for t in ([x] if c["mode"] != "col" else []) + ([x.t()] if c["mode"] != "row" else []):
        v, sc = _exact_codes(t, "e2m1")
        out.append(((v.view(*sc.shape, 32) * _two(sc.int() - 127)[..., None]).view(v.shape), sc))
    return out


def _exact_gemm4(c, s):
    return _exact_values(s["a"], s["sa"], c["a_elem"]) @ _exact_values(s["b"], s["sb"], "e2m1").t()


def _exact_grouped4(c, s):
    a, off = _exact_values(s["a"], s["sa"], c["a_elem"]), s["offsets"].tolist()
    rows = [a[off[g]:off[g + 1]] @ _exact_values(s["b"][g], s["sb"][g], "e2m1").t()
            for g in range(c["G"])]
    return torch.cat(rows)


# Results that are quantised after a computation stand beside the unrounded
# value over the block's scale, as 16-bit results do; their scale has no value
# in 64 bits where a block's largest magnitude lies next to a power's border.

def _over_scale(x, elem):
    e = _exact_scale(x.to(torch.bfloat16).double(), elem)
    return (x.reshape(*e.shape, 32) / _two(e)[..., None]).view(x.shape)


def _exact_swiglu(c, s):
    x = s["gate_up"].double()
    gate, up = x.split(c["F"], 1)
    out = [_over_scale(up * (gate * torch.sigmoid(gate)), c["elem"]), None]
    return out + list(_exact_codes(x, "e4m3")) if c["checkpoint"] else out


def _exact_swiglu_backward(c, s):
    gate, up = _exact_values(s["q"], s["s"], "e4m3").split(c["F"], 1)
    dh, p = s["dh"].double(), torch.sigmoid(gate)
    silu = gate * p
    d = torch.cat([dh * up * (p + silu * (1 - p)), dh * silu], 1)
    return d if c["elem"] == "bf16" else (_over_scale(d, c["elem"]), None)


def _exact_requant(c, s):
    x = _exact_values(s["q"], s["s"], c["elem"])
    if not c["G"]:
        return _exact_codes(x.t(), c["out_elem"])
    off = s["offsets"].tolist()
    cap = 128 * (c["T"] // 128 + c["G"])
    v = torch.zeros((c["C"], cap), dtype=torch.float64, device=x.device)
    sc = torch.zeros((c["C"], cap // 32), dtype=torch.uint8, device=x.device)
    for g in range(c["G"]):
        n = off[g + 1] - off[g]
        if n:
            at = 128 * (off[g] // 128 + g)
            part = torch.nn.functional.pad(x[off[g]:off[g + 1]].t(), (0, -n % 32))
            codes, scales = _exact_codes(part, c["out_elem"])
            v[:, at:at + n] = codes[:, :n]
            sc[:, at // 32:at // 32 + scales.shape[1]] = scales
    return v, sc


_EXACT = dict(quant4=_exact_quant4, gemm4=_exact_gemm4, grouped4=_exact_grouped4,
              swiglu=_exact_swiglu, swiglu_backward=_exact_swiglu_backward, requant=_exact_requant)
