"""Gradient norm and clipping on the GPU against the plain 64-bit
implementation, within derived bounds."""
import numpy as np
import pytest
import torch

import mxfp8_microscaled_precision_amd as mx
import plain_moe as P
from parity import host, say

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24                      # half a step of FP32, relative
HALF_BF16 = 2.0 ** -8


def _tensors(sizes, seed, std=0.01):
    g = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        t = std * torch.randn(n, generator=g)
        out.append(t.to(torch.bfloat16) if i % 3 else t)
    return out


def _check(ts, max_norm, dev_ts=None):
    """norm: sums in 64 bits, one rounding.  Clipped: the norm's, the sum's
    and the quotient's roundings in the coefficient, one for the product, one
    to the type."""
    t64 = [t.double().numpy() for t in ts]
    ref, scaled = P.grad_clip(t64, max_norm)
    d = [t.cuda() for t in ts] if dev_ts is None else dev_ts
    norm = mx.grad_norm(d)
    assert norm.shape == () and norm.dtype == torch.float32
    if ref < np.finfo(np.float32).max:
        assert abs(float(norm) - ref) <= 2 * EPS * ref
    else:
        assert float(norm) == np.inf          # rounded to FP32
    got = mx.grad_clip(d, max_norm)
    assert float(got) == float(norm)
    for t, g, want in zip(ts, d, scaled):
        tol = 6 * EPS * np.abs(want)
        if t.dtype == torch.bfloat16:
            tol = tol + HALF_BF16 * (np.abs(want) + tol) + 2.0 ** -134
        assert (np.abs(g.double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("sizes", [
    [1], [7], [0, 5, 0], [8192], [8191, 8193], [16384, 16385, 3], [1000003], [64] * 50,
    [1 + 37 * i for i in range(400)], [5] * 161, [300000, 17, 90001],
])
@pytest.mark.parametrize("share", [0.1, 0.999, 5.0])
def test_norm_and_clip(sizes, share):
    ts = _tensors(sizes, len(sizes))
    ref = P.grad_clip([t.double().numpy() for t in ts], 1.0)[0]
    _check(ts, float(np.float32(share * ref)))


def test_shapes_and_alignment():
    """Matrices, and tensors that start off 16 bytes."""
    flat = _tensors([5000, 5000, 5000, 5000], 1)
    ts, d = [], []
    for i, t in enumerate(flat):
        buf = torch.zeros(t.numel() + 8, dtype=t.dtype, device="cuda")
        v = buf[1 + i:1 + i + 4000].view(40, 100)
        v.copy_(t[:4000].view(40, 100))
        ts.append(t[:4000].view(40, 100))
        d.append(v)
    _check(ts, 0.05, d)


def test_nothing_outside_the_tensors_is_touched():
    buf = torch.ones(3 * 20000, dtype=torch.bfloat16, device="cuda")
    mid = buf[20003:39998]
    mx.grad_clip([mid], 1.0)
    got = host(buf.float())
    assert (got[:20003] == 1).all() and (got[39998:] == 1).all()
    assert (got[20003:39998] < 0.1).all()


def test_empty_lists():
    assert float(mx.grad_norm([])) == 0.0
    assert float(mx.grad_clip([], 1.0)) == 0.0
    assert float(mx.grad_clip([torch.empty(0, device="cuda")], 1.0)) == 0.0
    z = torch.zeros(10, device="cuda")
    assert float(mx.grad_clip([z], 0.0)) == 0.0 and (host(z) == 0).all()


def test_large_and_small_values():
    """Squares that pass FP32's range at either end."""
    ts = [torch.full((1000,), 3e37), torch.full((1000,), 2e37).to(torch.bfloat16)]
    _check(ts, 1.0)
    ts = [torch.full((1000,), 1e-30), torch.full((3,), 1e-30).to(torch.bfloat16)]
    norm = mx.grad_norm([t.cuda() for t in ts])
    ref = P.grad_clip([t.double().numpy() for t in ts], 1.0)[0]
    assert abs(float(norm) - ref) <= 2 * EPS * ref


def test_infinities_and_nan():
    t = torch.ones(100, device="cuda")
    t[3] = float("inf")
    norm = mx.grad_clip([t], 1.0)
    assert float(norm) == float("inf")
    got = host(t)
    assert np.isnan(got[3]) and (np.delete(got, 3) == 0).all()
    u = torch.ones(100, device="cuda", dtype=torch.bfloat16)
    u[50] = float("nan")
    v = torch.ones(5, device="cuda")
    assert np.isnan(float(mx.grad_clip([v, u], 1.0)))
    assert np.isnan(host(v)).all() and np.isnan(host(u.float())).all()


def test_max_norm_zero_and_repeatability():
    ts = [t.cuda() for t in _tensors([100000, 50001, 77], 5)]
    a = [float(mx.grad_norm(ts)) for _ in range(3)]
    assert a[0] == a[1] == a[2]
    mx.grad_clip(ts, 0.0)
    assert all((t == 0).all() for t in ts)


def test_gigabytes():
    """Offsets past 32 bits: one tensor of 2^31 + 5 BF16 elements."""
    n = (1 << 31) + 5
    t = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    t[-1] = 3.0
    ref = np.sqrt(0.25 * (n - 1) + 9.0)
    norm = mx.grad_clip([t], float(ref) / 4)
    assert abs(float(norm) - ref) <= 2 * EPS * ref
    assert float(t[0]) == 0.125 and float(t[n - 2]) == 0.125 and float(t[n - 1]) == 0.75
    assert int((t[:-1] != 0.125).sum()) == 0
    say("[grad] 4 GiB clipped")


def test_refusals():
    a = torch.zeros(100, device="cuda")
    for call, kind in [
        (lambda: mx.grad_norm([a.half()]), TypeError), (lambda: mx.grad_norm([a.view(10, 10).t()]), ValueError),
        (lambda: mx.grad_clip([a, a], 1.0), mx.MXError), (lambda: mx.grad_clip([a[:60], a[50:]], 1.0), mx.MXError),
        (lambda: mx.grad_clip([a], -1.0), mx.MXError), (lambda: mx.grad_clip([a], float("nan")), mx.MXError),
    ]:
        with pytest.raises(kind):
            call()
    mx.grad_norm([a, a])              # reading twice is no fault


def test_clipping_is_seen_by_autograd():
    """Scaling a tensor that a backward pass has saved makes that pass raise,
    as for any write in place; reading its norm does not.  Tensors of
    inference mode have no version and are clipped as they are."""
    t = torch.full((100,), 2.0, device="cuda")
    u = torch.full((40000,), 2.0, device="cuda").to(torch.bfloat16)
    w = torch.ones((100,), device="cuda", requires_grad=True)
    loss = (w * t).sum()
    versions = t._version, u._version
    mx.grad_norm([t, u])
    assert (t._version, u._version) == versions
    mx.grad_clip([t, u], 1.0)
    assert t._version > versions[0] and u._version > versions[1]
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
    with torch.inference_mode():
        free = torch.full((100,), 2.0, device="cuda")
    assert float(mx.grad_clip([free], 1.0)) == 20.0
    assert (free < 2.0).all()
