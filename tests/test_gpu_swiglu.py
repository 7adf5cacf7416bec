"""SwiGLU with a quantised result and an 8-bit checkpoint, and its gradient
from the checkpoint, on the GPU against the plain 64-bit reference."""
import numpy as np
import pytest
import torch

import mxfp8_microscaled_precision_amd as mx
import oracle
import plain_mx4 as P
from parity import assert_bytes, bits, dev, host

pytestmark = pytest.mark.gpu


def _x(T, F, seed, std=2.0):
    g = torch.Generator().manual_seed(seed)
    return (std * torch.randn((T, 2 * F), generator=g)).clamp(-16, 16).to(torch.bfloat16)


SHAPES = [(1, 32), (1, 18432), (2, 64), (7, 96), (33, 416), (129, 2048), (1000, 160), (3, 9216)]


@pytest.mark.parametrize("T,F", SHAPES)
@pytest.mark.parametrize("elem,ckpt", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2"),
                                       ("e4m3", None)])
def test_forward(T, F, elem, ckpt):
    x = _x(T, F, T + F)
    if ckpt:
        q, s, c = mx.swiglu_quant(x.cuda(), elem, checkpoint_elem=ckpt)
        oq, os_ = oracle.quant_row(bits(x), elem=ckpt)
        assert_bytes(c[0], oq, "checkpoint payload")
        assert_bytes(c[1], os_, "checkpoint scales")
    else:
        q, s, c = mx.swiglu_quant(x.cuda(), elem, checkpoint=False)
        assert c is None
    h = P.swiglu(P.bf16_values(bits(x)))
    wq, ws = P.quant_rows(P.bf16_round(h), elem)
    # a block whose values all round to one BF16 within the FP32 error is exact
    sure = P.bf16_decided(h).reshape(T, F // 32, 32).all(-1)
    assert sure.mean() > 0.5
    q, s = host(q), host(s)
    np.testing.assert_array_equal(s[sure], ws[sure])
    np.testing.assert_array_equal(q.reshape(T, -1, 32)[sure], wq.reshape(T, -1, 32)[sure])
    # elsewhere a value stands within half a code's step of one that differs
    # by a BF16 step; the scale may be the next one
    assert np.abs(s.astype(int) - ws).max() <= 1
    bits_, low = P.FORMAT[elem][1:]
    step = np.ldexp(1.0, np.maximum(np.frexp(h)[1] - 1 - bits_, (low - bits_ + np.repeat(s, 32, 1).astype(int) - 127)))
    off = np.abs(P.values(q, s, elem) - h)
    assert (off <= 0.5 * step * (1 + 2.0 ** -6) + 2.0 ** -7 * np.abs(h)).all()


@pytest.mark.parametrize("T,F", SHAPES)
@pytest.mark.parametrize("ckpt", ["e4m3", "e5m2"])
def test_backward(T, F, ckpt):
    c = oracle.quant_row(bits(_x(T, F, T + 2 * F)), elem=ckpt)
    dh = (0.01 * torch.randn((T, F), generator=torch.Generator().manual_seed(F))).to(torch.bfloat16)
    got = P.bf16_values(bits(mx.swiglu_backward(dh.cuda(), dev(c[0]), dev(c[1]), ckpt)))
    x, d = P.values(*c, ckpt), P.bf16_values(bits(dh))
    off = np.abs(got - P.swiglu_backward(d, x))
    assert (off <= P.swiglu_backward_tolerance(d, x)).all()


@pytest.mark.parametrize("T,F", SHAPES)
@pytest.mark.parametrize("ckpt,elem", [("e4m3", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
def test_backward_quant_is_quant_of_backward(T, F, ckpt, elem):
    c = [dev(t) for t in oracle.quant_row(bits(_x(T, F, T + 3 * F)), elem=ckpt)]
    dh = (0.01 * torch.randn((T, F), generator=torch.Generator().manual_seed(F))).to(torch.bfloat16).cuda()
    q, s = mx.swiglu_backward_quant(dh, *c, elem, ckpt)
    wq, ws = mx.quant(mx.swiglu_backward(dh, *c, ckpt), "row", elem)
    assert torch.equal(q, wq) and torch.equal(s, ws)


def test_special_values():
    """Gates at the ends of the range, infinities and NaN stay in their block."""
    x = _x(8, 64, 4)
    x[0, :4] = torch.tensor([300.0, -300.0, 88.0, -88.0])
    x[1, 0], x[1, 64] = 3e38, 3e38                     # the product overflows
    x[2, 0] = float("nan")
    x[3, 64 + 40] = float("inf")
    x[4] = 0.0
    x[5, :64] = -3e38                                  # every gate closed
    q, s, c = mx.swiglu_quant(x.cuda())
    with np.errstate(all="ignore"):
        h = P.bf16_round(P.swiglu(P.bf16_values(bits(x))))
    wq, ws = P.quant_rows(h, "e4m3")
    got, want = P.values(host(q), host(s), "e4m3"), P.values(wq, ws, "e4m3")
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    assert np.isnan(got[1, :32]).all() and np.isfinite(got[1, 32:]).all()
    assert np.isnan(got[2, :32]).all() and np.isfinite(got[2, 32:]).all()
    assert np.isnan(got[3, 32:]).all() and np.isfinite(got[3, :32]).all()
    assert not got[4].any() and not got[5].any()
    fine = ~np.isnan(want)
    assert (np.abs(got - want)[fine] <= 2.0 ** -3 * np.abs(want[fine]) + 2.0 ** -9 * np.abs(h[np.isfinite(h)]).max()).all()
    # the gradient: finite wherever the checkpoint's block and the result are
    dx = mx.swiglu_backward(torch.full((8, 64), 0.5, dtype=torch.bfloat16, device="cuda"), *c)
    d = P.bf16_values(bits(dx))
    ck = P.values(host(c[0]), host(c[1]), "e4m3")
    bad = np.isnan(ck)[:, :64] | np.isnan(ck)[:, 64:]
    np.testing.assert_array_equal(np.isnan(d[:, :64]), bad)
    with np.errstate(all="ignore"):
        want = P.bf16_round(P.swiglu_backward(np.full((8, 64), 0.5), ck))
    fin = np.isfinite(want) & np.isfinite(d)
    assert (np.isfinite(want) == np.isfinite(d))[:, :64][~bad].all()
    assert (np.abs(d - want)[fin] <= 2.0 ** -7 * np.abs(want[fin]) + 2.0 ** -100).all()


def test_empty_and_refusals():
    q, s, c = mx.swiglu_quant(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))
    assert tuple(q.shape) == (0, 32) and tuple(c[1].shape) == (0, 2)
    assert mx.swiglu_backward(torch.empty((0, 32), dtype=torch.bfloat16, device="cuda"), *c).shape == (0, 64)
    x = _x(4, 32, 1).cuda()
    with pytest.raises(ValueError):
        mx.swiglu_quant(x[:, :63].contiguous())
    with pytest.raises(mx.MXError):
        mx.swiglu_quant(x[:, :48].contiguous())
    with pytest.raises(TypeError):
        mx.swiglu_quant(x.float())
    q, s, c = mx.swiglu_quant(x)
    dh = torch.zeros((4, 32), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        mx.swiglu_backward(dh[:3], *c)
    with pytest.raises(ValueError):
        mx.swiglu_backward(dh, c[0], c[1][:, :1].contiguous())


def test_two_graphs_and_streams():
    x, dh = _x(40, 96, 8).cuda(), (0.1 * _x(40, 48, 9)).cuda()
    want = mx.swiglu_quant(x)
    dx = mx.swiglu_backward(dh, *want[2])
    dq = mx.swiglu_backward_quant(dh, *want[2])
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q, s, c = mx.swiglu_quant(x)
            outs = (q, s, *c, mx.swiglu_backward(dh, *c), *mx.swiglu_backward_quant(dh, *c))
        graphs.append((g, outs))
    for _ in range(3):
        for g, outs in graphs:
            for t in outs:
                t.zero_()
            g.replay()
        torch.cuda.synchronize()
        for g, outs in graphs:
            for a, b in zip(outs, (want[0], want[1], *want[2], dx, *dq)):
                assert torch.equal(a, b)
