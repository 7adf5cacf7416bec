"""The example's MoE training step: its results and gradients against its
formulas in 64 bits, a HIP graph of its calls, and a short training run."""
import os
import sys

import pytest
import torch

import mxfp8_microscaled_precision_amd as mx
import plain_moe as P
from parity import say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_training_step as M  # noqa: E402

pytestmark = pytest.mark.gpu


def _bf(t):
    return t.float().to(torch.bfloat16).double()


def _mx(t, dim):
    """t as MXFP8 holds it: blocks of 32 along dim (the last one may be short)
    share the smallest power of two that keeps them within 448."""
    t = t.transpose(0, dim)
    out = torch.empty_like(t)
    for i in range(0, t.shape[0], 32):
        b = t[i:i + 32]
        amax = b.abs().amax(0).clamp(min=2.0 ** -133)
        mant, e = torch.frexp(amax / 448.0)
        scale = torch.ldexp(torch.ones_like(amax), torch.where(mant == 0.5, e - 1, e))
        out[i:i + 32] = (b / scale).float().to(torch.float8_e4m3fn).double() * scale
    return out.transpose(0, dim)


def _reference(x, params, r, dout):
    """The step's formulas in 64 bits, expert by expert, with the operands and
    results rounded where the library holds MXFP8 and BF16."""
    c = {k: v.double().cpu() for k, v in params.items()}
    x, dout, e = x.double().cpu(), dout.double().cpu(), r.experts.cpu().long()
    logits = x @ c["router"].t()
    s = torch.sigmoid(logits)
    u = s.gather(1, e)
    w = u / u.sum(1, keepdim=True)
    out, dx = x.clone(), dout.clone()
    dw = torch.zeros_like(w)
    grads = {k: torch.zeros_like(c[k]) for k in ("gate_up", "down")}
    for i in range(c["router"].shape[0]):
        t, j = (e == i).nonzero(as_tuple=True)
        if len(t) == 0:
            continue
        gu_w, dn_w, wt = c["gate_up"][i], c["down"][i], w[t, j][:, None]
        gu = _bf(_mx(x[t], 1) @ _mx(gu_w, 1).t())
        gate, up = gu.chunk(2, 1)
        sig = torch.sigmoid(gate)
        h = _bf(gate * sig * up)
        y = _bf(_mx(h, 1) @ _mx(dn_w, 1).t())
        out.index_add_(0, t, wt * y)
        dw[t, j] = (dout[t] * y).sum(1)
        dy = _bf(wt * dout[t])
        dh = _bf(_mx(dy, 1) @ _mx(dn_w, 0))
        dgu = _bf(torch.cat([dh * up * sig * (1 + gate * (1 - sig)), dh * gate * sig], 1))
        dx.index_add_(0, t, _bf(_mx(dgu, 1) @ _mx(gu_w, 0)))
        grads["gate_up"][i] = _mx(dgu, 0).t() @ _mx(x[t], 0)
        grads["down"][i] = _mx(dy, 0).t() @ _mx(h, 0)
    dl = torch.from_numpy(P.route_backward(dw.numpy(), logits.numpy(), e.numpy(), "sigmoid", True, 1.0))
    grads["router"] = dl.t() @ x
    return out, _bf(dx) + dl @ c["router"], grads


def test_step_matches_its_formulas():
    """Against the same formulas in 64 bits.  Both sides round to MXFP8 and
    BF16 at the same places, from values that differ by the GPU's 32-bit sums
    alone; those move a BF16 rounding (2^-8) of few elements, and one in 16 of
    these an E4M3 rounding (2^-3) of the next operand: well under 2^-8 of a
    product's norm, and the last BF16 rounding as much again.  2^-6 over the
    chain of up to four products."""
    T, H, F, E, k = 96, 128, 64, 8, 2
    params = M.init(H, F, E, 3)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    dout = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    out, _, dx, grads, norm, r = M.step(x, params, lambda o: (0.0, dout), k, 4, 2, max_norm=1e9)
    rout, rdx, rgrads = _reference(x, params, r, dout)

    def far(a, b):
        return float((a.double().cpu() - b).norm() / b.norm())

    dist = {"out": far(out, rout), "dx": far(dx, rdx), **{n: far(grads[n], rgrads[n]) for n in grads}}
    say("[moe step]", {n: round(v, 5) for n, v in dist.items()})
    assert all(v < 2.0 ** -6 for v in dist.values()), dist
    want = sum(float(t.double().square().sum()) for t in grads.values()) ** 0.5
    assert abs(float(norm) - want) <= 2.0 ** -22 * want


def test_training_lowers_the_loss():
    losses = M.train(steps=4, T=512, H=256, F=128, E=8, top_k=2, say=say)
    assert all(b < a for a, b in zip(losses, losses[1:]))


def test_captured_calls_replay_as_eager():
    """Every new entry point in one HIP graph, replayed three times with its
    outputs overwritten and other eager work in between."""
    g = torch.Generator(device="cuda").manual_seed(5)
    T, E, k, H = 700, 64, 6, 520
    logits = torch.randn((T, E), generator=g, device="cuda")
    logits[::9] = -float("inf")
    bias = 0.1 * torch.randn((E,), generator=g, device="cuda")
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    xq = torch.randn((T, 544), generator=g, device="cuda").to(torch.bfloat16)
    y = torch.randn((T * k, H), generator=g, device="cuda").to(torch.bfloat16)
    fresh = [torch.randn((n,), generator=g, device="cuda").to(t) for n, t in
             ((100000, torch.bfloat16), (33333, torch.float32), (5, torch.bfloat16))] * 70
    fresh = [t.clone() for t in fresh]
    grads = [t.clone() for t in fresh]

    def calls():
        r = mx.route(logits, k, "sigmoid", bias, n_groups=8, top_groups=4)
        q, s = mx.dispatch_quant(xq, r)
        out = mx.combine(y, r, residual=x)
        dy, dw = mx.combine_backward(x, y, r)
        dl = mx.route_backward(dw, logits, r.experts, "sigmoid")
        for t, f in zip(grads, fresh):
            t.copy_(f)
        norm = mx.grad_clip(grads, 1.0)
        return [*r, mx.dispatch(x, r), q, s, out, dy, dw, dl, norm, mx.grad_norm(grads[:3]), *grads]

    eager = [t.clone() for t in calls()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls()
    for rep in range(3):
        for t in outs:
            t.fill_(0x5A if not t.is_floating_point() else float("nan"))
        mx.route(logits[:100].contiguous(), k)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, eager)):
            assert torch.equal(a, b), (rep, i)
    say("[graph] three replays equal the eager run")
