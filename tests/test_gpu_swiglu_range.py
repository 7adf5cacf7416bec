"""SwiGLU and its gradient at the ends of their range: the widest rows and the
largest magnitudes."""
import pytest
import torch

import mxfp8_microscaled_precision_amd as mx

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
