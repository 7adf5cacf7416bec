"""4-bit quantisation, restoring and column blocks from row blocks on the GPU,
byte for byte against the plain 64-bit reference and the oracle."""
import numpy as np
import pytest
import torch

import mxfp8_microscaled_precision_amd as mx
import oracle
import plain_mx4 as P
from parity import assert_bytes, bits, dev, host

pytestmark = pytest.mark.gpu


def _bf16(shape, seed, spread=2.0):
    """Normal values whose rows and columns differ in magnitude, with zero
    blocks, ties of the 4-bit grid and the ends of the range among them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    x = x * torch.exp(spread * torch.randn(shape[:-1] + (1,), generator=g))
    x = x * torch.exp(0.5 * torch.randn(shape[-1:], generator=g))
    flat = x.view(-1)
    n = flat.numel()
    for i, v in enumerate([0.25, -0.75, 2.5, 5.0, 6.0, -6.0, 6.03125, 3.0, 0.0, -0.0, 3.3e38, 1e-39, 2.0 ** -133]):
        flat[(97 * i + 13) % n] = v
    return x.to(torch.bfloat16)


def _special(rows, cols, seed):
    x = _bf16((rows, cols), seed, 1.0)
    x[0] = 0.0
    x[1, 5] = float("nan")
    x[2, cols - 1] = float("-inf")
    x[3] = torch.tensor([1], dtype=torch.int16).view(torch.bfloat16)[0]     # smallest subnormal
    x[4, ::3] = 3.38e38
    x[:, cols - 2] = 0.0
    return x


def _want(x, mode):
    v = P.bf16_values(bits(x))
    out = []
    if mode != "col":
        out += P.quant_rows(v, "e2m1")
    if mode != "row":
        out += P.quant_rows(np.ascontiguousarray(np.swapaxes(v, -1, -2)), "e2m1")
    return out


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (1, 18432), (1021, 416), (32, 32), (64, 96), (96, 64),
                                       (256, 64), (288, 160), (512, 128), (544, 1056), (1024, 32), (32, 2080)])
@pytest.mark.parametrize("mode", ["row", "col", "dual"])
def test_quant4(rows, cols, mode):
    if mode != "row" and rows % 32:
        with pytest.raises(mx.MXError):
            mx.quant4(torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda"), mode)
        return
    x = _bf16((rows, cols), rows + cols)
    for got, want in zip(mx.quant4(x.cuda(), mode), _want(x, mode)):
        assert_bytes(got, want, f"{mode} [{rows}, {cols}]")


@pytest.mark.parametrize("mode", ["row", "col", "dual"])
def test_quant4_special_values(mode):
    for rows, cols in ((32, 64), (320, 192)):
        x = _special(rows, cols, 5)
        for got, want in zip(mx.quant4(x.cuda(), mode), _want(x, mode)):
            assert_bytes(got, want, mode)


@pytest.mark.parametrize("mode", ["row", "col", "dual"])
@pytest.mark.parametrize("B,rows,cols", [(1, 32, 64), (3, 288, 96), (5, 64, 160)])
def test_quant4_stack(B, rows, cols, mode):
    x = _bf16((B, rows, cols), B)
    for got, want in zip(mx.quant4(x.cuda(), mode), _want(x, mode)):
        assert_bytes(got, want, mode)


def test_quant4_every_bf16_against_every_scale_neighbour():
    """All 65536 patterns in blocks of their own neighbours."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(2048, 32)
    q, s = mx.quant4(x.cuda(), "row")
    wq, ws = _want(x, "row")
    assert_bytes(q, wq, "payload")
    assert_bytes(s, ws, "scales")


def test_quant4_empty():
    for shape in ((0, 64), (32, 0), (0, 32, 64)):
        for mode in ("row", "col", "dual"):
            for t in mx.quant4(torch.empty(shape, dtype=torch.bfloat16, device="cuda"), mode):
                assert t.numel() == 0


@pytest.mark.parametrize("elem", ["e4m3", "e5m2", "e2m1"])
def test_dequant_every_code_at_every_scale(elem):
    codes = np.tile(np.arange(16 if elem == "e2m1" else 256, dtype=np.uint8), (256, 2))
    s = np.repeat(np.arange(256, dtype=np.uint8)[:, None], codes.shape[1] // 32, 1)
    q = P.pack(codes) if elem == "e2m1" else codes
    got = P.bf16_values(bits(mx.dequant(dev(q), dev(s), elem)))
    want = P.bf16_round(P.values(q, s, elem))
    np.testing.assert_array_equal(got, want)
    np.testing.assert_array_equal(np.signbit(got[~np.isnan(got)]), np.signbit(want[~np.isnan(want)]))


@pytest.mark.parametrize("elem", ["e4m3", "e5m2", "e2m1"])
@pytest.mark.parametrize("shape", [(1, 32), (7, 96), (1021, 416), (2, 3, 64), (18432,)])
def test_dequant_shapes(elem, shape):
    rng = np.random.default_rng(len(shape))
    q = rng.integers(0, 256, shape[:-1] + (shape[-1] // (2 if elem == "e2m1" else 1),), dtype=np.uint8)
    s = rng.integers(100, 150, shape[:-1] + (shape[-1] // 32,), dtype=np.uint8)
    y = mx.dequant(dev(q), dev(s), elem)
    assert tuple(y.shape) == shape
    np.testing.assert_array_equal(P.bf16_values(bits(y)), P.values(q, s, elem))


@pytest.mark.parametrize("elem", ["e4m3", "e5m2"])
@pytest.mark.parametrize("out_elem", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,cols", [(32, 32), (64, 160), (128, 128), (288, 96), (1056, 416)])
def test_requant_col(rows, cols, elem, out_elem):
    x = _special(rows, cols, rows) if rows > 64 else _bf16((rows, cols), rows)
    q, s = mx.quant(x.cuda(), "row", elem)
    qt, st = mx.requant_col(q, s, elem, out_elem)
    restored = P.to_bf16_bits(P.bf16_round(P.values(host(q), host(s), elem)))
    wq, ws = oracle.quant_col(restored, elem=out_elem)
    assert_bytes(qt, wq, "payload")
    assert_bytes(st, ws, "scales")
    two = mx.quant(mx.dequant(q, s, elem), "col", out_elem)
    assert torch.equal(two[0], qt) and torch.equal(two[1], st)


OFFSETS = [[0, 5], [0, 0, 37, 37, 100, 128], [0, 128, 256, 300], [0, 1, 2, 3, 3, 200], [0, 129, 130, 131, 1000],
           [0, 0, 0], [0, 33]]


@pytest.mark.parametrize("off", OFFSETS)
@pytest.mark.parametrize("elem,out_elem", [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
def test_requant_grouped_col(off, elem, out_elem):
    T, C = off[-1], 160
    off = np.array(off, np.int64)
    x = _bf16((T, C), T + 1) if T else torch.empty((0, C), dtype=torch.bfloat16)
    q, s = mx.quant(x.cuda(), "row", elem)
    qt, st = mx.requant_grouped_col(q, s, dev(off), elem, out_elem)
    if T:
        restored = P.to_bf16_bits(P.bf16_round(P.values(host(q), host(s), elem)))
        wq, ws = oracle.quant_col_grouped(restored, off, elem=out_elem)
        assert_bytes(qt, wq, "payload")
        assert_bytes(st, ws, "scales")
    else:
        assert not host(qt).any() and not host(st).any()


def test_requant_grouped_col_with_bad_offsets_stays_in_bounds():
    """Offsets past the rows, negative or decreasing: wrong blocks, but every
    output is written and nothing else is read."""
    q, s = mx.quant(_bf16((96, 64), 9).cuda(), "row")
    for off in ([0, 500, 96], [-40, 30, 96], [0, 90, 20, 96], [7, 7, 7, 1 << 60]):
        qt, st = mx.requant_grouped_col(q, s, dev(np.array(off, np.int64)))
        assert tuple(qt.shape) == (64, mx.grouped_col_capacity(96, len(off) - 1))


def test_strided_and_misaligned_tensors_are_refused():
    x = _bf16((64, 128), 1).cuda()
    with pytest.raises(ValueError, match="contiguous"):
        mx.quant4(x.t(), "row")
    with pytest.raises(ValueError, match="contiguous"):
        mx.quant4(x[:, :64], "row")
    odd = torch.zeros(64 * 128 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(64, 128)
    with pytest.raises(mx.MXError, match="aligned"):
        mx.quant4(odd, "row")
    q, s = mx.quant4(x, "row")
    with pytest.raises(ValueError):
        mx.dequant(q, s[:, :3], "e2m1")
    with pytest.raises(ValueError):
        mx.dequant(q, s, "e4m3")


def test_four_bit_calls_on_another_stream_and_in_a_graph():
    x = _bf16((288, 192), 3).cuda()
    want = mx.quant4(x, "dual")
    back = mx.dequant(want[0], want[1], "e2m1")
    q8, s8 = mx.quant(x, "row")
    cols = mx.requant_col(q8, s8)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = mx.quant4(x, "dual")
        y = mx.dequant(got[0], got[1], "e2m1")
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(y, back)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = mx.quant4(x, "dual")
        outs = (*out, mx.dequant(out[0], out[1], "e2m1"), *mx.requant_col(q8, s8))
    for _ in range(3):
        for t in outs:
            t.zero_()
        graph.replay()
        (x.float() * 2).sum().item()               # the program's own work between replays
        for a, b in zip(outs, (*want, back, *cols)):
            assert torch.equal(a, b)
