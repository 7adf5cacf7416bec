"""One training step of an MoE layer from this library's calls.

    python examples/moe_training_step.py [mxfp8|mxfp4]

A token batch is routed to its experts, dispatched into the expert order in
MXFP8, run through the experts' two products with a SwiGLU between them and
combined back onto the residual stream; the backward pass gives the gradients
of the input, the expert weights and the router, which are clipped together.
``step`` is the layer; ``train`` trains a small one for a few steps and prints
loss, expert load and gradient norm.  PyTorch does the router's product, the
SwiGLU of the 8-bit form and the weight update.

With ``mxfp4`` the experts' weights are used in 4 bits (the BF16 copies stay the
ones that are trained: the gradient passes the rounding as it is), the SwiGLU
is the library's, and what the backward pass needs of the activations is kept
in 8 bits: the products' row-quantised operands and the gate/up checkpoint.
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


def _experts8(x, r, params):
    """The experts' MLP on dispatched rows with MXFP8 weights: its result, and
    the backward pass that turns the result's gradient into the rows' and the
    weights'."""
    w_gu, w_dn = params["gate_up"], params["down"]
    qx, sx = mx.dispatch_quant(x, r)
    gu = mx.grouped_gemm(r.offsets, qx, sx, *mx.quant_batched(w_gu, "row"))
    h, saved = _swiglu(gu)
    y = mx.grouped_gemm(r.offsets, *mx.quant(h, "row"), *mx.quant_batched(w_dn, "row"))

    def backward(dy):
        dh = mx.grouped_gemm(r.offsets, *mx.quant(dy, "row"), *mx.quant_batched(w_dn, "col"))
        dgu = _swiglu_backward(dh, saved)
        dxe = mx.grouped_gemm(r.offsets, *mx.quant(dgu, "row"), *mx.quant_batched(w_gu, "col"))
        rows = r.slots.numel()
        xe = mx.dispatch(x, r)
        return dxe, {
            "gate_up": mx.grouped_gemm_wgrad(r.offsets, rows, *mx.quant_grouped_col(dgu, r.offsets),
                                             *mx.quant_grouped_col(xe, r.offsets)),
            "down": mx.grouped_gemm_wgrad(r.offsets, rows, *mx.quant_grouped_col(dy, r.offsets),
                                          *mx.quant_grouped_col(h, r.offsets)),
        }

    return y, backward


def _experts4(x, r, params):
    """The same with 4-bit weights; between the passes the rows, the SwiGLU's
    result and its gates and up values are held in 8 bits."""
    gu4, gu4_s, gu4_t, gu4_ts = mx.quant4(params["gate_up"], "dual")
    dn4, dn4_s, dn4_t, dn4_ts = mx.quant4(params["down"], "dual")
    qx, sx = mx.dispatch_quant(x, r)
    gu = mx.grouped_gemm4(r.offsets, qx, sx, gu4, gu4_s)
    qh, sh, ckpt = mx.swiglu_quant(gu)
    y = mx.grouped_gemm4(r.offsets, qh, sh, dn4, dn4_s)

    def backward(dy):
        dh = mx.grouped_gemm4(r.offsets, *mx.quant(dy, "row"), dn4_t, dn4_ts)
        qd, sd = mx.swiglu_backward_quant(dh, *ckpt)
        dxe = mx.grouped_gemm4(r.offsets, qd, sd, gu4_t, gu4_ts)
        rows = r.slots.numel()
        return dxe, {
            "gate_up": mx.grouped_gemm_wgrad(r.offsets, rows, *mx.requant_grouped_col(qd, sd, r.offsets),
                                             *mx.requant_grouped_col(qx, sx, r.offsets)),
            "down": mx.grouped_gemm_wgrad(r.offsets, rows, *mx.quant_grouped_col(dy, r.offsets),
                                          *mx.requant_grouped_col(qh, sh, r.offsets)),
        }

    return y, backward


EXPERTS = {"mxfp8": _experts8, "mxfp4": _experts4}


def step(x, params, dout_of, top_k, n_groups=1, top_groups=1, max_norm=1.0, weights="mxfp8"):
    """x BF16 [T, H]; params: router FP32 [E, H], bias FP32 [E], gate_up BF16
    [E, 2F, H], down BF16 [E, H, F]; dout_of(out) -> (loss, gradient of out);
    weights: the experts' ("mxfp8" or "mxfp4").

    Returns (out, loss, dx, gradients by name, norm before clipping, routing).
    """
    # forward
    logits = x.float() @ params["router"].t()
    r = mx.route(logits, top_k, "sigmoid", params["bias"], n_groups=n_groups, top_groups=top_groups)
    y, experts_backward = EXPERTS[weights](x, r, params)
    out = mx.combine(y, r, residual=x)
    loss, dout = dout_of(out)

    # backward: through combine, the experts, dispatch, and the router
    dy, dweights = mx.combine_backward(dout, y, r)
    dxe, grads = experts_backward(dy)
    dlogits = mx.route_backward(dweights, logits, r.experts, "sigmoid")
    dx = mx.combine(dxe, r, residual=dout, weighted=False).float() + dlogits @ params["router"]
    grads["router"] = dlogits.t() @ x.float()
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


def train(steps=8, T=2048, H=512, F=256, E=16, top_k=4, lr=1.0, say=print, weights="mxfp8"):
    params = init(H, F, E)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    target = torch.randn((T, H), generator=g, device="cuda")

    def mse(out):
        d = out.float() - target
        return (d * d).mean(), (2.0 / d.numel() * d).to(torch.bfloat16)

    losses = []
    for i in range(steps):
        _, loss, _, grads, norm, r = step(x, params, mse, top_k, n_groups=4, top_groups=2, weights=weights)
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
    train(weights=sys.argv[1] if len(sys.argv) > 1 else "mxfp8")
