"""One training step of an MoE layer from this library's calls.

    python examples/moe_training_step.py

A token batch is routed to its experts, dispatched into the expert order in
MXFP8, run through the experts' two products with a SwiGLU between them and
combined back onto the residual stream; the backward pass gives the gradients
of the input, the expert weights and the router, which are clipped together.
``step`` is the layer; ``main`` trains a small one for a few steps and prints
loss, expert load and gradient norm.  PyTorch does the router's product, the
SwiGLU and the weight update.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp8_microscaled_precision_amd as mx  # noqa: E402


def _swiglu(gu):
    """h = silu(gate) * up, and what its gradient needs."""
    gate, up = gu.float().chunk(2, dim=1)
    sig = torch.sigmoid(gate)
    return (gate * sig * up).to(torch.bfloat16), (gate, up, sig)


def _swiglu_backward(dh, saved):
    gate, up, sig = saved
    dh = dh.float()
    dgate = dh * up * sig * (1.0 + gate * (1.0 - sig))
    return torch.cat([dgate, dh * gate * sig], dim=1).to(torch.bfloat16)


def step(x, params, dout_of, top_k, n_groups=1, top_groups=1, max_norm=1.0):
    """x BF16 [T, H]; params: router FP32 [E, H], bias FP32 [E], gate_up BF16
    [E, 2F, H], down BF16 [E, H, F]; dout_of(out) -> (loss, gradient of out).

    Returns (out, loss, dx, gradients by name, norm before clipping, routing).
    """
    w_gu, w_dn = params["gate_up"], params["down"]

    # forward
    logits = x.float() @ params["router"].t()
    r = mx.route(logits, top_k, "sigmoid", params["bias"], n_groups=n_groups, top_groups=top_groups)
    qx, sx = mx.dispatch_quant(x, r)
    gu = mx.grouped_gemm(r.offsets, qx, sx, *mx.quant_batched(w_gu, "row"))
    h, saved = _swiglu(gu)
    y = mx.grouped_gemm(r.offsets, *mx.quant(h, "row"), *mx.quant_batched(w_dn, "row"))
    out = mx.combine(y, r, residual=x)
    loss, dout = dout_of(out)

    # backward: through combine, the down product, the SwiGLU, the gate_up
    # product, dispatch, and the router
    dy, dweights = mx.combine_backward(dout, y, r)
    dh = mx.grouped_gemm(r.offsets, *mx.quant(dy, "row"), *mx.quant_batched(w_dn, "col"))
    dgu = _swiglu_backward(dh, saved)
    dxe = mx.grouped_gemm(r.offsets, *mx.quant(dgu, "row"), *mx.quant_batched(w_gu, "col"))
    dlogits = mx.route_backward(dweights, logits, r.experts, "sigmoid")
    dx = mx.combine(dxe, r, residual=dout, weighted=False).float() + dlogits @ params["router"]

    rows = r.slots.numel()
    xe = mx.dispatch(x, r)
    grads = {
        "gate_up": mx.grouped_gemm_wgrad(r.offsets, rows, *mx.quant_grouped_col(dgu, r.offsets),
                                         *mx.quant_grouped_col(xe, r.offsets)),
        "down": mx.grouped_gemm_wgrad(r.offsets, rows, *mx.quant_grouped_col(dy, r.offsets),
                                      *mx.quant_grouped_col(h, r.offsets)),
        "router": dlogits.t() @ x.float(),
    }
    norm = mx.grad_clip(list(grads.values()), max_norm)
    return out, loss, dx.to(torch.bfloat16), grads, norm, r


def init(H, F, E, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device=device)  # noqa: E731
    return {
        "router": rand(E, H) * H ** -0.5,
        "bias": torch.zeros(E, device=device),
        "gate_up": (rand(E, 2 * F, H) * H ** -0.5).to(torch.bfloat16),
        "down": (rand(E, H, F) * F ** -0.5).to(torch.bfloat16),
    }


def train(steps=8, T=2048, H=512, F=256, E=16, top_k=4, lr=1.0, say=print):
    params = init(H, F, E)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    target = torch.randn((T, H), generator=g, device="cuda")

    def mse(out):
        d = out.float() - target
        return (d * d).mean(), (2.0 / d.numel() * d).to(torch.bfloat16)

    losses = []
    for i in range(steps):
        _, loss, _, grads, norm, r = step(x, params, mse, top_k, n_groups=4, top_groups=2)
        load = torch.diff(r.offsets).float()
        for name, d in grads.items():
            params[name] -= (lr * d.float()).to(params[name].dtype)
        # the balance bias rises for experts with less than their share
        params["bias"] += 0.01 * torch.sign(load.mean() - load)
        losses.append(float(loss))
        say(f"step {i}: loss {losses[-1]:.4f}  gradient norm {float(norm):.4f}  "
            f"largest expert {int(load.max())} of {int(load.sum())} choices")
    return losses


if __name__ == "__main__":
    torch.cuda.set_device(0)
    train()
