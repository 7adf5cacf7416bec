"""Dispatch and combine on the GPU: copied and quantised rows byte for byte,
sums and gradients against the plain 64-bit implementation within derived
bounds."""
import numpy as np
import pytest
import torch

import mxfp8_microscaled_precision_amd as mx
import oracle
import plain_moe as P
from parity import assert_bytes, bits, dev, host, say

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24                      # half a step of FP32, relative
HALF_BF16 = 2.0 ** -8


def _routing(T, E, k, seed, drop=0.0):
    rng = np.random.default_rng(seed)
    e = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    e[rng.random(e.shape) < drop] = -1
    off, slots = P.layout(e, E)
    w = np.where(e < 0, 0.0, rng.random(e.shape)).astype(np.float32)
    return mx.Routing(dev(w), dev(e), dev(off), dev(slots)), off, slots, w


def _bf16(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (std * torch.randn(shape, generator=g)).to(torch.bfloat16)


SHAPES = [(1, 1, 1, 32), (1, 64, 8, 7168), (3, 8, 2, 1), (5, 4, 4, 7), (17, 60, 6, 1000), (64, 64, 8, 512),
          (70, 16, 3, 513), (33, 512, 16, 520), (100, 8, 8, 4096), (257, 60, 5, 96), (9, 10, 9, 2050),
          (2000, 64, 2, 64), (40, 64, 8, 2048)]


@pytest.mark.parametrize("T,E,k,H", SHAPES)
@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
def test_dispatch(T, E, k, H, drop):
    r, _, slots, _ = _routing(T, E, k, T + H, drop)
    x = _bf16((T, H), H)
    y = mx.dispatch(x.cuda(), r)
    want = P.dispatch(bits(x), slots)
    np.testing.assert_array_equal(bits(y), want)
    if H % 32 == 0:
        for elem in ("e4m3", "e5m2"):
            q, s = mx.dispatch_quant(x.cuda(), r, elem)
            oq, os_ = oracle.quant_row(want, elem=elem)
            assert_bytes(q, oq, f"{elem} payload")
            assert_bytes(s, os_, f"{elem} scales")


def test_dispatch_quant_special_values():
    """Blocks of NaN, Inf, zeros and subnormals, as the row quantiser has them."""
    x = _bf16((12, 128), 3)
    x[0] = 0.0
    x[1, 5] = float("nan")
    x[2, 40] = float("inf")
    x[3] = torch.tensor([1], dtype=torch.int16).view(torch.bfloat16)[0]     # smallest subnormal
    x[4, ::7] = 3e38
    r, _, slots, _ = _routing(12, 6, 3, 1, 0.2)
    for elem in ("e4m3", "e5m2"):
        q, s = mx.dispatch_quant(x.cuda(), r, elem)
        oq, os_ = oracle.quant_row(P.dispatch(bits(x), slots), elem=elem)
        used = int((slots >= 0).sum())
        assert_bytes(q[:used], oq[:used], "payload")
        assert_bytes(s[:used], os_[:used], "scales")
        gq, gs = mx.quant(mx.dispatch(x.cuda(), r), "row", elem)
        assert torch.equal(q, gq) and torch.equal(s, gs)


@pytest.mark.parametrize("T,E,k,H", SHAPES)
@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
def test_combine(T, E, k, H, drop):
    r, _, slots, w = _routing(T, E, k, T + H + 1, drop)
    y, res = _bf16((T * k, H), H + 1), _bf16((T, H), H + 2)
    y64 = y.double().numpy()
    for weighted in (True, False):
        for residual in (None, res):
            got = mx.combine(y.cuda(), r, None if residual is None else residual.cuda(), weighted)
            ref, mag = P.combine(y64, slots, w.astype(np.float64) if weighted else None,
                                 None if residual is None else residual.double().numpy())
            # k products and sums in FP32, one rounding to BF16
            tol = (k + 2) * EPS * mag
            tol = tol + HALF_BF16 * (np.abs(ref) + tol)
            assert (np.abs(got.double().cpu().numpy() - ref) <= tol).all()
    out = res.cuda()
    assert torch.equal(mx.combine(y.cuda(), r, out, out=out), mx.combine(y.cuda(), r, res.cuda()))


def _dot_tol(H, mag):
    # a lane adds at most 8 products of each of its spans, then lanes and
    # waves are added in at most 6 + 16 steps
    return (8 * -(-H // 512) + 24) * EPS * mag


@pytest.mark.parametrize("T,E,k,H", SHAPES)
@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
def test_combine_backward(T, E, k, H, drop):
    r, _, slots, w = _routing(T, E, k, T + H + 2, drop)
    y, d = _bf16((T * k, H), H + 3), _bf16((T, H), H + 4, 0.01)
    dy, dw = mx.combine_backward(d.cuda(), y.cuda(), r)
    rdy, rdw, mag = P.combine_backward(d.double().numpy(), y.double().numpy(), slots,
                                       w.astype(np.float64))
    # one FP32 product, one rounding to BF16
    tol = (HALF_BF16 + 2 * EPS) * np.abs(rdy) + 2.0 ** -134
    assert (np.abs(dy.double().cpu().numpy() - rdy) <= tol).all()
    assert (np.abs(host(dw) - rdw) <= _dot_tol(H, mag) + 1e-44).all()


def test_combine_backward_matches_differences():
    """The GPU's weight gradient against central differences of the 64-bit
    sums (which are linear in the weights)."""
    r, _, slots, w = _routing(4, 6, 3, 8)
    y, d = _bf16((12, 40), 1), _bf16((4, 40), 2)
    _, dw = mx.combine_backward(d.cuda(), y.cuda(), r)
    y64, d64, w64 = y.double().numpy(), d.double().numpy(), w.astype(np.float64)
    mag = P.combine_backward(d64, y64, slots, w64)[2]
    for i in np.ndindex(4, 3):
        h = np.zeros_like(w64)
        h[i] = 0.5
        diff = ((P.combine(y64, slots, w64 + h)[0] - P.combine(y64, slots, w64 - h)[0]) * d64).sum()
        assert abs(diff - float(dw[i])) <= _dot_tol(40, mag[i]) + 1e-10


def test_combine_is_dispatch_gradient():
    """<dispatch(x), dy> = <x, combine(dy, unweighted)>."""
    r, _, slots, _ = _routing(50, 16, 4, 9, 0.2)
    x, dy = _bf16((50, 72), 5), _bf16((200, 72), 6)
    dx = mx.combine(dy.cuda(), r, weighted=False).double().cpu().numpy()
    y = mx.dispatch(x.cuda(), r).double().cpu().numpy()
    lhs, rhs = (y * dy.double().numpy()), (x.double().numpy() * dx)
    _, mag = P.combine(dy.double().numpy(), slots)
    tol = ((HALF_BF16 + 6 * EPS) * mag * np.abs(x.double().numpy())).sum()
    assert abs(lhs.sum() - rhs.sum()) <= tol


@pytest.mark.parametrize("H", [64, 100])
def test_operands_off_16_byte_alignment(H):
    r, _, slots, w = _routing(30, 8, 3, 4, 0.1)
    x, y, res = _bf16((30, H), 1), _bf16((90, H), 2), _bf16((30, H), 3)

    def off(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        v = flat[1:].view(t.shape)
        v.copy_(t)
        return v

    assert torch.equal(mx.dispatch(off(x), r), mx.dispatch(x.cuda(), r))
    assert torch.equal(mx.combine(off(y), r, off(res), out=off(res)), mx.combine(y.cuda(), r, res.cuda()))
    a, b = mx.combine_backward(off(x), off(y), r)
    c, d = mx.combine_backward(x.cuda(), y.cuda(), r)
    assert torch.equal(a, c)
    mag = P.combine_backward(x.double().numpy(), y.double().numpy(), slots, w.astype(np.float64))[2]
    assert (np.abs(host(b).astype(np.float64) - host(d)) <= 2 * _dot_tol(H, mag)).all()
    if H % 32 == 0:
        for p, q in zip(mx.dispatch_quant(off(x), r), mx.dispatch_quant(x.cuda(), r)):
            assert torch.equal(p, q)


def test_bad_slots_are_skipped():
    """Slots outside the rows and a wild offset touch nothing out of bounds."""
    r, _, slots, w = _routing(20, 8, 2, 4)
    bad = slots.copy()
    bad[3, 0], bad[5, 1], bad[7, 0] = 40, 1 << 30, -7
    clean = np.where((bad < 0) | (bad >= 40), -1, bad)
    rb = r._replace(slots=dev(bad))
    rc = r._replace(slots=dev(clean))
    x, y = _bf16((20, 64), 1), _bf16((40, 64), 2)
    taken = sorted(int(v) for v in clean[clean >= 0])
    assert torch.equal(mx.dispatch(x.cuda(), rb)[taken], mx.dispatch(x.cuda(), rc)[taken])
    assert torch.equal(mx.dispatch_quant(x.cuda(), rb)[0][taken], mx.dispatch_quant(x.cuda(), rc)[0][taken])
    assert torch.equal(mx.combine(y.cuda(), rb), mx.combine(y.cuda(), rc))
    got, want = mx.combine_backward(x.cuda(), y.cuda(), rb), mx.combine_backward(x.cuda(), y.cuda(), rc)
    assert torch.equal(got[0][taken], want[0][taken]) and torch.equal(got[1], want[1])
    for wild in (-5, 1 << 40):
        o = r.offsets.clone()
        o[-1] = wild
        mx.dispatch(x.cuda(), r._replace(offsets=o))
    torch.cuda.synchronize()


def test_no_token_and_empty_rows():
    r, _, _, _ = _routing(4, 8, 2, 1)
    e = mx.Routing(*(t[:0] if t.dim() == 2 else t * 0 for t in r))
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    assert mx.dispatch(x, e).shape == (0, 64) and mx.combine(x, e).shape == (0, 64)
    dy, dw = mx.combine_backward(x, x, e)
    assert dy.shape == (0, 64) and dw.shape == (0, 2)
    z = torch.empty((4, 0), dtype=torch.bfloat16, device="cuda")
    zz = torch.empty((8, 0), dtype=torch.bfloat16, device="cuda")
    assert mx.dispatch(z, r).shape == (8, 0)
    assert (host(mx.combine_backward(z, zz, r)[1]) == 0).all()


def test_rows_past_2_31_bytes():
    """Rows whose byte offsets pass 32 bits are reached."""
    T, k, H = 1 << 16, 8, 4224                     # 4.4 GB of expert rows
    g = torch.Generator(device="cuda").manual_seed(1)
    slots = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32).view(T, k)
    r = mx.Routing(torch.full((T, k), 0.125, device="cuda"), slots,
                   torch.arange(k + 1, device="cuda") * T, slots)
    x = torch.randn((T, 1), generator=g, device="cuda").to(torch.bfloat16).expand(T, H).contiguous()
    y = mx.dispatch(x, r)
    src = torch.empty(T * k, dtype=torch.int64, device="cuda")
    src[slots.flatten().long()] = torch.arange(T * k, device="cuda") // k
    assert torch.equal(y[:, 0], x[src, 0]) and torch.equal(y[:, H - 1], x[src, 0])
    assert torch.equal(mx.combine(y, r), x)        # eight eighths
    dy, dw = mx.combine_backward(x, y, r)
    assert torch.equal(dy[:, H - 1], (x[src, 0].float() * 0.125).to(torch.bfloat16))
    q, s = mx.dispatch_quant(x, r)
    rq, rs = mx.quant(x, "row")
    assert torch.equal(q[:, H - 1], rq[src, H - 1]) and torch.equal(s[:, -1], rs[src, -1])
    say("[move] 4.4 GB of expert rows")


def test_refusals():
    r, _, _, _ = _routing(4, 8, 2, 1)
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")
    for call, kind in [
        (lambda: mx.dispatch(x[:3], r), ValueError), (lambda: mx.dispatch(x.float(), r), TypeError),
        (lambda: mx.dispatch(x.t(), r), ValueError),
        (lambda: mx.dispatch(x, r._replace(slots=r.slots.long())), TypeError),
        (lambda: mx.dispatch(x, r._replace(offsets=r.offsets[:1])), ValueError),
        (lambda: mx.dispatch_quant(x[:, :40].contiguous(), r), mx.MXError),
        (lambda: mx.combine(x, r), ValueError), (lambda: mx.combine(y, r, y), ValueError),
        (lambda: mx.combine(y, r, out=y), ValueError),
        (lambda: mx.combine(y, r._replace(weights=r.weights[:3])), ValueError),
        (lambda: mx.combine_backward(y, y, r), ValueError),
        (lambda: mx.combine_backward(x, x, r), ValueError),
    ]:
        with pytest.raises(kind):
            call()


def test_combine_refuses_an_output_that_shares_memory():
    """With one choice y and out have one shape, and views overlap in part."""
    r, _, _, _ = _routing(4, 8, 1, 1)
    buf = torch.zeros((6, 64), dtype=torch.bfloat16, device="cuda")
    y, res = buf[:4], torch.zeros((5, 64), dtype=torch.bfloat16, device="cuda")
    for call in (lambda: mx.combine(y, r, out=y), lambda: mx.combine(y, r, out=buf[2:]),
                 lambda: mx.combine(y, r, res[:4], out=res[1:])):
        with pytest.raises(mx.MXError, match="shares memory"):
            call()
    mx.combine(y[:4], r, res[:4], out=res[:4])
    two = torch.zeros((8, 64), dtype=torch.bfloat16, device="cuda")       # neighbours do not overlap
    mx.combine(two[:4], r, out=two[4:])


def test_combine_into_a_tensor_is_seen_by_autograd():
    """Writing into a tensor that a backward pass has saved makes that pass
    raise, as for any write in place; tensors of inference mode have no
    version and are taken as they are."""
    r, _, _, _ = _routing(4, 8, 2, 1)
    y, out = _bf16((8, 64), 1).cuda(), torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    loss = (w * out).sum()
    version = out._version
    want = mx.combine(y, r)
    assert torch.equal(mx.combine(y, r, out=out), want)
    assert out._version > version
    with pytest.raises(RuntimeError, match="inplace"):
        loss.backward()
    with torch.inference_mode():
        free = torch.zeros_like(out)
    assert torch.equal(mx.combine(y, r, out=free), want)


def test_choices_dropped_and_numbered_anew():
    """A choice taken out of slots alone leaves the rows of the others as they
    are; numbered anew, the rows that are left over are zero."""
    r, _, slots, w = _routing(50, 8, 2, 4)
    x, y = _bf16((50, 64), 1), _bf16((100, 64), 2)
    e = host(r.experts).copy()
    e[::7, 1] = -1
    holes = np.where(e < 0, -1, slots)
    named = holes[holes >= 0]
    want = P.dispatch(bits(x), holes)
    got = bits(mx.dispatch(x.cuda(), r._replace(slots=dev(holes))))
    np.testing.assert_array_equal(got[named], want[named])
    off, anew = P.layout(e, 8)
    rr = mx.Routing(dev(np.where(e < 0, 0.0, w).astype(np.float32)), dev(e), dev(off), dev(anew))
    np.testing.assert_array_equal(bits(mx.dispatch(x.cuda(), rr)), P.dispatch(bits(x), anew))
    used = int(off[-1])
    q, s = mx.dispatch_quant(x.cuda(), rr)
    dy, dw = mx.combine_backward(x.cuda(), y.cuda(), rr)
    assert used == named.size < 100
    assert not host(q[used:]).any() and not host(s[used:]).any() and not host(dy[used:].float()).any()
    assert (host(dw)[e < 0] == 0).all()


@pytest.mark.parametrize("T,k,H", [(20000, 8, 2048), (41001, 8, 992), (26011, 3, 4224)])
@pytest.mark.parametrize("elem", ["e4m3", "e5m2"])
def test_dispatch_quant_past_the_cache(T, k, H, elem):
    """Payloads of over 300 MiB, rows in whole lines and not: the
    bytes of quantising the dispatched rows, and zeros past them."""
    g = torch.Generator(device="cuda").manual_seed(H)
    e = torch.rand((T, 16), generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32)
    e[::5, k - 1] = -1
    off, slots = P.layout(host(e), 16)
    r = mx.Routing(torch.zeros((T, k), device="cuda"), e.contiguous(), dev(off), dev(slots))
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    q, s = mx.dispatch_quant(x, r, elem)
    y = mx.dispatch(x, r)
    rq, rs = mx.quant(y, "row", elem)
    assert torch.equal(q, rq) and torch.equal(s, rs)
    assert not q[int(off[-1]):].any()
