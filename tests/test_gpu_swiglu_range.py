"""SwiGLU and its gradient at the ends of their range: the widest rows and the
largest magnitudes."""
import numpy as np
import pytest
import torch

import mxfp8_microscaled_precision_amd as mx
import plain_mx4 as P
from parity import bits, dev, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("F", [(1 << 32) + 64, (1 << 33) - 32])
def test_rows_past_32_bit_columns(F):
    """Columns past 2^32 are their own: every stretch of a row has the bytes of
    a short row of the same values."""
    n = 128
    spans = [0, (1 << 31) - n // 2, (1 << 32) - n // 2, F - n]
    g = torch.Generator(device="cuda").manual_seed(1)

    def cut(t, at):                               # columns at .. at + n - 1 of both halves
        return torch.cat([t[:, at:at + n], t[:, F + at:F + at + n]], 1)

    x = torch.empty((1, 2 * F), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    q, s, (cq, cs) = mx.swiglu_quant(x)
    short = {}
    for at in spans:
        wq, ws, ck = short[at] = mx.swiglu_quant(cut(x, at))
        assert torch.equal(q[:, at:at + n], wq) and torch.equal(s[:, at // 32:(at + n) // 32], ws)
        assert torch.equal(cut(cq, at), ck[0])
        scales = torch.cat([cs[:, at // 32:(at + n) // 32], cs[:, (F + at) // 32:(F + at + n) // 32]], 1)
        assert torch.equal(scales, ck[1])
    del x, q, s
    dh = torch.empty((1, F), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    dx = mx.swiglu_backward(dh, cq, cs)
    for at in spans:
        want = mx.swiglu_backward(dh[:, at:at + n].contiguous(), *short[at][2])
        assert torch.equal(cut(dx, at).view(torch.int16), want.view(torch.int16))
    del dx
    q, s = mx.swiglu_backward_quant(dh, cq, cs)
    for at in spans:
        wq, ws = mx.swiglu_backward_quant(dh[:, at:at + n].contiguous(), *short[at][2])
        assert torch.equal(cut(q, at), wq)
        scales = torch.cat([s[:, at // 32:(at + n) // 32], s[:, (F + at) // 32:(F + at + n) // 32]], 1)
        assert torch.equal(scales, ws)


# FP32 evaluation for gates down to -168: the exponent's argument, below 256 in
# powers of two, carries half a step of its product (2^-17) and the constant's
# own rounding (2^-16), which the exponential turns into as much of its value;
# the other operations add 2^-23 each.  Together under 2^-14.
DEEP_EPS = 2.0 ** -14


def _deep_gates():
    """Rows of one gate each, with up values that bring the result back into
    BF16's normal range: [rows, 32] gates, [rows, 32] up values."""
    rng = np.random.default_rng(3)
    gates = np.array([-64.0, -79.5, -80.0, -80.5, -84.0, -87.0, -87.5, -88.0, -88.5, -96.0, -104.0, -120.0, -144.0, -166.0])
    g = np.repeat(gates[:, None], 32, 1)
    u = (1 + rng.random(g.shape)) * np.ldexp(1.0, np.clip(np.rint(-g * 1.4427), 0, 126).astype(int)) \
        * np.where(rng.random(g.shape) < 0.5, -1, 1)
    return P.bf16_round(g), P.bf16_round(u)


def test_gates_whose_sigmoid_has_no_fp32_value():
    """Below -87 the sigmoid passes FP32's smallest normal value; times the up
    value the result does not."""
    g, u = _deep_gates()
    x = torch.from_numpy(np.concatenate([g, u], 1)).to(torch.bfloat16)
    q, s, _ = mx.swiglu_quant(x.cuda())
    h = P.swiglu(np.concatenate([g, u], 1))
    assert (np.abs(h) > 2.0 ** -126).all()
    # half a step of E4M3 and of BF16, and the smallest code of the block
    floor = np.ldexp(1.0, np.repeat(host(s), 32, 1).astype(int) - 127 - 10)
    off = np.abs(P.values(host(q), host(s), "e4m3") - h)
    assert (off <= (2.0 ** -4 + 2.0 ** -7 + DEEP_EPS) * np.abs(h) + floor).all()


@pytest.mark.parametrize("elem", ["e4m3", "e5m2"])
def test_gradient_at_gates_whose_sigmoid_has_no_fp32_value(elem):
    g, u = _deep_gates()
    x = np.concatenate([g, u], 1)
    ck = P.quant_rows(x, elem)
    x = P.values(*ck, elem)
    # one half row has dh near 1, the other brings du into the normal range
    for dh in (np.ones_like(g), P.bf16_round(np.abs(u))):
        if dh[0, 0] != 1:
            x = x.copy()
            x[:, 32:] = P.bf16_round(np.sign(x[:, 32:]))
            ck = P.quant_rows(x, elem)
        got = P.bf16_values(bits(mx.swiglu_backward(torch.from_numpy(dh).to(torch.bfloat16).cuda(),
                                                    dev(ck[0]), dev(ck[1]), elem)))
        ref = P.swiglu_backward(dh, x)
        p = P.sigmoid(x[:, :32])
        mag = np.concatenate([np.abs(dh * x[:, 32:]) * p * (1 + np.abs(x[:, :32])), np.abs(dh * x[:, :32]) * p], 1)
        assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + DEEP_EPS * mag + 2.0 ** -133).all()


def test_closed_gates_of_any_size_give_zero():
    """Gates from -200 to the type's lowest value, up values and gradients to its
    largest: zeros, no NaN (but where the checkpoint holds an infinity: E4M3 rounds
    the largest BF16 values to 2^128)."""
    big = float(torch.finfo(torch.bfloat16).max)
    gate = torch.tensor([-200.0, -1e4, -1e20, -1e38], dtype=torch.bfloat16).repeat_interleave(32).view(4, 32)
    up = torch.tensor([1.0, -3e38, big, -1e-30], dtype=torch.bfloat16).repeat(8).expand(4, 32)
    x = torch.cat([gate, up], 1).contiguous().cuda()
    q, s, ck = mx.swiglu_quant(x)
    assert not (host(q) & 0x7F).any() and not host(s).any()
    finite = torch.isfinite(mx.dequant(*ck)[:, 32:])
    assert finite.float().mean() > 0.7
    finite = torch.cat([finite, torch.ones_like(finite)], 1)
    for d in (1.0, 3e38):
        dx = mx.swiglu_backward(torch.full((4, 32), d, dtype=torch.bfloat16, device="cuda"), *ck).float()
        assert (dx[finite] == 0).all()


def test_gradient_where_up_values_near_the_end_meet_small_gradients():
    """p (1 + g (1 - p)) passes 1 for gates above 1.28: times an up value near the
    type's end it leaves FP32's range, the gradient's own value does not."""
    rng = np.random.default_rng(5)
    g = P.bf16_round(rng.uniform(1.5, 4.0, (8, 32)))
    u = np.full((8, 32), 1.875 * 2.0 ** 127) * np.where(rng.random((8, 32)) < 0.5, -1, 1)
    ck = P.quant_rows(np.concatenate([g, u], 1), "e4m3")
    x = P.values(*ck, "e4m3")
    assert (np.abs(x[:, 32:]) == 1.875 * 2.0 ** 127).all()
    for scale in (1e-2, 1e-20, 0.9):
        dh = P.bf16_round(scale * rng.uniform(0.5, 1.0, (8, 32)))
        got = P.bf16_values(bits(mx.swiglu_backward(torch.from_numpy(dh).to(torch.bfloat16).cuda(), dev(ck[0]), dev(ck[1]))))
        ref = P.swiglu_backward(dh, x)
        assert (np.abs(got - ref) <= P.swiglu_backward_tolerance(dh, x)).all()


@pytest.mark.parametrize("elem", ["e4m3", "e5m2"])
def test_rows_do_not_depend_on_far_neighbours(elem):
    """A wave with gates below -80 or up values near 2^128 takes another form: its
    other rows have the bits that they have alone, products below FP32's normal
    range among them."""
    rng = np.random.default_rng(9)
    T, F = 512, 32
    g = rng.uniform(-70, 70, (T, F))
    u = rng.uniform(1, 2, (T, F)) * np.ldexp(1.0, rng.integers(-126, 126, (T, 1)))
    dh = rng.uniform(1, 2, (T, F)) * np.ldexp(1.0, rng.integers(-126, 126, (T, 1)))
    x = torch.from_numpy(np.concatenate([g, u], 1)).to(torch.bfloat16).cuda()
    dh = torch.from_numpy(dh).to(torch.bfloat16).cuda()
    far = torch.full((T, 2 * F), -96.0, dtype=torch.bfloat16, device="cuda")
    far[::2] = 3.3e38
    both = torch.stack([x, far], 1).view(2 * T, 2 * F)
    d2 = torch.stack([dh, dh], 1).view(2 * T, F)
    one, two = mx.swiglu_quant(x, checkpoint_elem=elem), mx.swiglu_quant(both, checkpoint_elem=elem)
    assert torch.equal(one[0], two[0][::2]) and torch.equal(one[1], two[1][::2])
    a, b = mx.swiglu_backward(dh, *one[2], elem), mx.swiglu_backward(d2, *two[2], elem)
    assert torch.equal(a.view(torch.int16), b[::2].contiguous().view(torch.int16))
