"""The 4-bit and checkpoint calls together, as an MLP's training step and a
decoding step use them: a dense MLP stage by stage, the example's MoE step with
4-bit weights against its formulas in 64 bits, and captured graphs."""
import os
import sys

import numpy as np
import pytest
import torch

import mxfp8_microscaled_precision_amd as mx
import oracle
import plain_moe
import plain_mx4 as P
from parity import bits, dev, host, say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import moe_training_step as M  # noqa: E402

pytestmark = pytest.mark.gpu


def _bf16(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (std * torch.randn(shape, generator=g)).to(torch.bfloat16)


def _bits4(x, mode):
    v = P.bf16_values(bits(x))
    return P.quant_rows(v if mode == "row" else np.ascontiguousarray(v.T), "e2m1")


def _near(got, ref, absum, K, elem, what):
    off = np.abs(P.bf16_values(bits(got)) - ref)
    assert (off <= P.gemm_tolerance(ref, absum, K, elem)).all(), what


@pytest.mark.parametrize("T", [1, 33, 160])
def test_dense_mlp_forward_and_backward_stage_by_stage(T):
    """Every product against the 64-bit one of the operands it was given, every
    quantised operand byte for byte where its input is known in bits."""
    H, F = 160, 96
    x, w_gu, w_dn = _bf16((T, H), 1), _bf16((2 * F, H), 2, 0.1), _bf16((H, F), 3, 0.1)
    dy = _bf16((T, H), 4, 0.1)
    qx, sx = mx.quant(x.cuda(), "row")
    gu4, gu4_s, gu4_t, gu4_ts = mx.quant4(w_gu.cuda(), "dual")
    dn4, dn4_s, dn4_t, dn4_ts = mx.quant4(w_dn.cuda(), "dual")
    gu = mx.gemm4(qx, sx, gu4, gu4_s)
    ax = oracle.quant_row(bits(x))
    _near(gu, *P.gemm(*ax, *_bits4(w_gu, "row"), "e4m3"), H, "e4m3", "gate_up")
    qh, sh, ckpt = mx.swiglu_quant(gu)
    h = P.swiglu(P.bf16_values(bits(gu)))
    ah = host(qh), host(sh)
    # E4M3 of a BF16 of h: half a step of each, and the block's smallest step
    floor = np.ldexp(1.0, np.repeat(ah[1], 32, 1).astype(int) - 127 - 10)
    assert (np.abs(P.values(*ah, "e4m3") - h) <= (2.0 ** -4 + 2.0 ** -7) * np.abs(h) + floor).all()
    y = mx.gemm4(qh, sh, dn4, dn4_s)
    _near(y, *P.gemm(*ah, *_bits4(w_dn, "row"), "e4m3"), F, "e4m3", "down")
    # backward
    qd, sd = mx.quant(dy.cuda(), "row")
    dh = mx.gemm4(qd, sd, dn4_t, dn4_ts)
    _near(dh, *P.gemm(*oracle.quant_row(bits(dy)), *_bits4(w_dn, "col"), "e4m3"), H, "e4m3", "dh")
    dgu = mx.swiglu_backward(dh, *ckpt)
    c, d = P.values(host(ckpt[0]), host(ckpt[1]), "e4m3"), P.bf16_values(bits(dh))
    assert (np.abs(P.bf16_values(bits(dgu)) - P.swiglu_backward(d, c)) <= P.swiglu_backward_tolerance(d, c)).all()
    qg, sg = mx.swiglu_backward_quant(dh, *ckpt)
    dx = mx.gemm4(qg, sg, gu4_t, gu4_ts)
    ag = host(qg), host(sg)
    _near(dx, *P.gemm(*ag, *_bits4(w_gu, "col"), "e4m3"), 2 * F, "e4m3", "dx")
    if T % 32 == 0:
        # weight gradients from the 8-bit row blocks that the forward pass kept
        def cols(q, s):
            v = P.to_bf16_bits(P.bf16_round(P.values(host(q), host(s), "e4m3")))
            return oracle.quant_col(v)
        for (qa, sa), (qb, sb) in (((qg, sg), (qx, sx)), ((qd, sd), (qh, sh))):
            at, bt = mx.requant_col(qa, sa), mx.requant_col(qb, sb)
            dw = mx.gemm(*at, *bt, "wgrad")
            ref, bound = oracle.gemm(*cols(qa, sa), *cols(qb, sb))
            assert oracle.within_tolerance(P.bf16_values(bits(dw)), ref, bound).all()


def _bf(t):
    return t.float().to(torch.bfloat16).double()


def _mx(t, dim, elem="e4m3"):
    """t as an MX tensor holds it, blocks of 32 along dim (a short last one
    padded with zeros, which change no maximum)."""
    v = np.ascontiguousarray(t.transpose(dim, -1).numpy())
    n = v.shape[-1]
    pad = np.pad(v, [(0, 0)] * (v.ndim - 1) + [(0, -n % 32)])
    return torch.from_numpy(P.values(*P.quant_rows(pad, elem), elem)[..., :n].copy()).transpose(dim, -1)


def _reference(x, params, r, dout):
    """The step's formulas in 64 bits, expert by expert, rounded where the
    library holds 4 bits, 8 bits or BF16."""
    c = {k: v.double().cpu() for k, v in params.items()}
    x, dout, e = x.double().cpu(), dout.double().cpu(), r.experts.cpu().long()
    logits = x @ c["router"].t()
    u = torch.sigmoid(logits).gather(1, e)
    w = u / u.sum(1, keepdim=True)
    out, dx = x.clone(), dout.clone()
    dw = torch.zeros_like(w)
    grads = {k: torch.zeros_like(c[k]) for k in ("gate_up", "down")}
    for i in range(c["router"].shape[0]):
        t, j = (e == i).nonzero(as_tuple=True)
        if len(t) == 0:
            continue
        gu_w, dn_w, wt = c["gate_up"][i], c["down"][i], w[t, j][:, None]
        x8 = _mx(x[t], 1)
        gu = _bf(x8 @ _mx(gu_w, 1, "e2m1").t())
        h8 = _mx(_bf(torch.from_numpy(P.swiglu(gu.numpy()))), 1)
        y = _bf(h8 @ _mx(dn_w, 1, "e2m1").t())
        out.index_add_(0, t, wt * y)
        dw[t, j] = (dout[t] * y).sum(1)
        dy = _bf(wt * dout[t])
        dh = _bf(_mx(dy, 1) @ _mx(dn_w, 0, "e2m1"))
        dgu = _bf(torch.from_numpy(P.swiglu_backward(dh.numpy(), _mx(gu, 1).numpy())))
        d8 = _mx(dgu, 1)
        dx.index_add_(0, t, _bf(d8 @ _mx(gu_w, 0, "e2m1")))
        grads["gate_up"][i] = _mx(d8, 0).t() @ _mx(x8, 0)
        grads["down"][i] = _mx(dy, 0).t() @ _mx(h8, 0)
    dl = torch.from_numpy(plain_moe.route_backward(dw.numpy(), logits.numpy(), e.numpy(), "sigmoid", True, 1.0))
    grads["router"] = dl.t() @ x
    return out, _bf(dx) + dl @ c["router"], grads


def test_moe_step_with_4_bit_weights_matches_its_formulas():
    """Both sides round at the same places, from values that differ by the
    products' sums: 7 2^-13 of the magnitudes in the worst of cases (see
    gemm_tolerance) and some 2^-13 of the norm in the mean of terms of either
    sign, which moves a BF16 rounding (2^-8) of one element in 32 or fewer, and
    of these one in 16 an E4M3 rounding (2^-3 of it): 2^-3 sqrt(2^-9) < 2^-7 of an
    operand's norm, twice where it is rounded to 8 bits twice.  Over the chain of
    three products and up to five such operands 2^-7 sqrt(5) < 2^-5."""
    T, H, F, E, k = 96, 128, 64, 8, 2
    params = M.init(H, F, E, 3)
    x, dout = _bf16((T, H), 4).cuda(), _bf16((T, H), 5).cuda()
    out, _, dx, grads, norm, r = M.step(x, params, lambda o: (0.0, dout), k, 4, 2, max_norm=1e9, weights="mxfp4")
    rout, rdx, rgrads = _reference(x, params, r, dout)

    def far(a, b):
        return float((a.double().cpu() - b).norm() / b.norm())

    dist = {"out": far(out, rout), "dx": far(dx, rdx), **{n: far(grads[n], rgrads[n]) for n in grads}}
    say("[moe step, 4-bit weights]", {n: round(v, 5) for n, v in dist.items()})
    assert all(v < 2.0 ** -5 for v in dist.values()), dist


def test_example_runs_with_4_bit_weights():
    losses = M.train(steps=2, T=256, H=128, F=64, E=8, top_k=2, say=say, weights="mxfp4")
    assert len(losses) == 2 and all(np.isfinite(losses))


def test_eight_bit_form_of_the_example_is_as_before():
    """The 8-bit step is the calls that it was, in their order."""
    T, H, F, E, k = 96, 128, 64, 8, 2
    params = M.init(H, F, E, 3)
    x, dout = _bf16((T, H), 4).cuda(), _bf16((T, H), 5).cuda()
    out, _, _, grads, _, r = M.step(x, params, lambda o: (0.0, dout), k, max_norm=1e9)
    qx, sx = mx.dispatch_quant(x, r)
    gu = mx.grouped_gemm(r.offsets, qx, sx, *mx.quant_batched(params["gate_up"], "row"))
    h, _ = M._swiglu(gu)
    y = mx.grouped_gemm(r.offsets, *mx.quant(h, "row"), *mx.quant_batched(params["down"], "row"))
    assert torch.equal(out, mx.combine(y, r, residual=x))
    dy, _ = mx.combine_backward(dout, y, r)
    assert torch.equal(grads["down"], mx.grouped_gemm_wgrad(
        r.offsets, T * k, *mx.quant_grouped_col(dy, r.offsets), *mx.quant_grouped_col(h, r.offsets)))


def test_moe_step_in_a_graph_while_an_eager_one_lives():
    """The step's calls captured, replayed and run eagerly in turn, on one
    stream, give the eager bits every time."""
    T, H, F, E, k = 200, 128, 96, 8, 2
    params = M.init(H, F, E, 6)
    x, dy = _bf16((T, H), 7).cuda(), _bf16((T * k, H), 8).cuda()
    logits = torch.randn((T, E), generator=torch.Generator().manual_seed(9)).cuda()

    def calls():
        r = mx.route(logits, k)
        y, backward = M._experts4(x, r, params)
        dxe, grads = backward(dy)
        return [y, dxe, grads["gate_up"], grads["down"]]

    eager = [t.clone() for t in calls()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls()
    for _ in range(3):
        for t in outs:
            t.fill_(float("nan"))
        graph.replay()
        again = calls()
        for a, b, c in zip(outs, again, eager):
            assert torch.equal(a, c) and torch.equal(b, c)


def test_decoding_step_in_one_graph():
    """One token through a layer whose contraction is split over workgroups:
    two graphs side by side, each with its own partial sums."""
    H, F = 4096, 12288
    w = [mx.quant4(_bf16((n, k), i, 0.02).cuda()) for i, (n, k) in enumerate(((2 * 512, H), (512, F)))]
    x = [_bf16((1, H), 10 + i).cuda() for i in range(2)]
    z = [_bf16((1, F), 20 + i).cuda() for i in range(2)]

    def calls(i):
        gu = mx.gemm4(*mx.quant(x[i], "row"), *w[0])
        q, s, _ = mx.swiglu_quant(gu, checkpoint=False)
        return gu, q, s, mx.gemm4(*mx.quant(z[i], "row"), *w[1])

    assert mx.mx_gemm4_workspace_size(0, 1, 512, F) > 0
    want = [[t.clone() for t in calls(i)] for i in range(2)]
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = calls(i)
        graphs.append((g, outs))
    side = torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[1][0].replay()
        graphs[0][0].replay()
        torch.cuda.synchronize()
        for (_, outs), ref in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip(outs, ref))
