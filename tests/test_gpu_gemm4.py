"""Products with 4-bit weights on the GPU against the plain 64-bit reference,
within a bound derived from the FP32 sums and the BF16 rounding."""
import numpy as np
import pytest
import torch

import mxfp8_microscaled_precision_amd as mx
import plain_mx4 as P
from parity import bits, dev

pytestmark = pytest.mark.gpu

ELEMS = ["e4m3", "e5m2", "e2m1"]


def _operand(shape, elem, seed):
    """Codes of normal values, rows of differing magnitude."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(shape) * np.exp(rng.standard_normal(shape[:-1] + (1,)))
    return P.quant_rows(x, elem)


def _close(got, ref, absum, K, elem, what):
    got = P.bf16_values(bits(got))
    off, tol = np.abs(got - ref), P.gemm_tolerance(ref, absum, K, elem)
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, worst {np.nanmax(off / tol):.3g} at {np.argwhere(bad)[0]}"


def _check(M, N, K, elem, seed=0):
    a, sa = _operand((M, K), elem, seed + M)
    b, sb = _operand((N, K), "e2m1", seed + N + 1000)
    got = mx.gemm4(dev(a), dev(sa), dev(b), dev(sb), elem)
    _close(got, *P.gemm(a, sa, b, sb, elem), K, elem, f"{elem} {M} x {N} x {K}")


# every number of rows around a kernel's row tiles, odd and aligned columns
SHAPES = [(1, 1, 32), (1, 16, 64), (1, 33, 256), (1, 100, 288), (2, 32, 512), (3, 7, 2080), (15, 64, 544),
          (16, 130, 1024), (17, 48, 96), (31, 34, 2048), (32, 256, 1056), (33, 31, 768), (48, 260, 512),
          (63, 129, 288), (64, 128, 1280), (65, 64, 512), (100, 300, 480), (129, 258, 1024), (200, 64, 4096),
          (255, 255, 992), (256, 256, 512), (257, 260, 1536), (300, 514, 64), (513, 264, 2560), (1, 8, 18432),
          (5, 40, 32768)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("elem", ELEMS)
def test_gemm4(M, N, K, elem):
    _check(M, N, K, elem)


@pytest.mark.parametrize("elem", ELEMS)
def test_gemm4_many_tiles(elem):
    """More tiles than compute units; ragged in both directions."""
    _check(4100, 4360, 512, elem)
    _check(2300, 7432, 1024, elem)


@pytest.mark.parametrize("elem", ELEMS)
@pytest.mark.parametrize("N,K", [(3304, 128), (3301, 160), (3304, 544), (3303, 768), (3298, 1024), (3302, 2080)])
def test_gemm4_many_tiles_of_any_length(elem, N, K):
    """Rows that end inside a K step, inside a dword of scales, at every parity."""
    _check(3301, N, K, elem)


@pytest.mark.parametrize("elem", ELEMS)
@pytest.mark.parametrize("M", [1, 20, 300])
def test_one_hot_rows_give_the_weight(elem, M):
    """One code 1.0 a row: the result is a column of the weight, exactly, at
    every position of K; every lane and byte has its own."""
    N, K = 48, 1024
    b, sb = _operand((N, K), "e2m1", 5)
    w = P.values(b, sb, "e2m1")
    one = {"e4m3": 0x38, "e5m2": 0x3C, "e2m1": 2}[elem]
    for first in range(0, K, M):
        rows = np.arange(first, min(first + M, K))
        codes = np.zeros((len(rows), K), np.uint8)
        codes[np.arange(len(rows)), rows] = one
        a = P.pack(codes) if elem == "e2m1" else codes
        sa = np.full((len(rows), K // 32), 127, np.uint8)
        got = P.bf16_values(bits(mx.gemm4(dev(a), dev(sa), dev(b), dev(sb), elem)))
        np.testing.assert_array_equal(got, w[:, rows].T)
        if M == 1 and first >= 64:
            break


@pytest.mark.parametrize("elem", ELEMS)
@pytest.mark.parametrize("M,K", [(1, 1024), (3, 544), (300, 1024), (300, 544)])
def test_every_block_has_its_own_scale(elem, M, K):
    """Codes of one, scales that differ by block and row: exact sums of powers."""
    N = 40
    rng = np.random.default_rng(M + K)
    one = {"e4m3": 0x38, "e5m2": 0x3C, "e2m1": 2}[elem]
    codes = np.full((M, K), one, np.uint8)
    a = P.pack(codes) if elem == "e2m1" else codes
    b = P.pack(np.full((N, K), 2, np.uint8))
    sa = rng.integers(120, 130, (M, K // 32), dtype=np.uint8)
    sb = rng.integers(120, 130, (N, K // 32), dtype=np.uint8)
    got = P.bf16_values(bits(mx.gemm4(dev(a), dev(sa), dev(b), dev(sb), elem)))
    np.testing.assert_array_equal(got, P.bf16_round(P.gemm(a, sa, b, sb, elem)[0]))


@pytest.mark.parametrize("M", [2, 40, 300])
def test_not_a_number_scales_and_zeros(M):
    N, K = 70, 544
    a, sa = _operand((M, K), "e4m3", 1)
    b, sb = _operand((N, K), "e2m1", 2)
    sa[1, 3] = 255
    sb[5, 16] = 255
    b[6] = 0
    got = P.bf16_values(bits(mx.gemm4(dev(a), dev(sa), dev(b), dev(sb))))
    assert np.isnan(got[1]).all() and np.isnan(got[:, 5]).all()
    rows = [r for r in range(M) if r != 1]
    assert not got[rows, 6].any()
    rest = np.delete(np.delete(got, 1, 0), 5, 1)
    assert np.isfinite(rest).all()


def test_large_and_small_scales():
    """Products past FP32's range become infinite, tiny ones vanish; no NaN."""
    N, K = 33, 256
    one = np.full((4, K), 0x38, np.uint8)
    b = P.pack(np.full((N, K), 2, np.uint8))
    sb = np.full((N, K // 32), 254, np.uint8)
    sa = np.array([[254], [0], [127], [1]], np.uint8).repeat(K // 32, 1)
    got = P.bf16_values(bits(mx.gemm4(dev(one), dev(sa), dev(b), dev(sb))))
    assert np.isinf(got[0]).all() and (got[1] == K).all() and np.isinf(got[2]).all() and (got[3] == 2 * K).all()


def test_empty_products():
    u8 = dict(dtype=torch.uint8, device="cuda")
    z = mx.gemm4(torch.empty((3, 0), **u8), torch.empty((3, 0), **u8), torch.empty((5, 0), **u8),
                 torch.empty((5, 0), **u8))
    assert z.shape == (3, 5) and not z.float().any()
    assert mx.gemm4(torch.empty((0, 64), **u8), torch.empty((0, 2), **u8), torch.empty((5, 32), **u8),
                    torch.empty((5, 2), **u8)).shape == (0, 5)
    off = torch.zeros(3, dtype=torch.int64, device="cuda")
    assert mx.grouped_gemm4(off, torch.empty((0, 64), **u8), torch.empty((0, 2), **u8),
                            torch.empty((2, 5, 32), **u8), torch.empty((2, 5, 2), **u8)).shape == (0, 5)


GROUPS = [[0, 1], [0, 0, 3, 3, 8], [0, 1, 2, 3, 4, 5, 6, 7, 8], [0, 17, 17, 50, 64], [0, 100, 101, 200],
          [0, 256, 256, 700, 701], [0, 3, 600, 600, 1200], [0, 40, 80], [5, 20, 31]]


@pytest.mark.parametrize("off", GROUPS)
@pytest.mark.parametrize("elem", ELEMS)
@pytest.mark.parametrize("N,K", [(1, 32), (130, 288), (264, 1024)])
def test_grouped(off, elem, N, K):
    G, T = len(off) - 1, off[-1] + 4              # four rows behind the last group
    a, sa = _operand((T, K), elem, T)
    b, sb = _operand((G, N, K), "e2m1", N)
    out = torch.full((T, N), -3.0, dtype=torch.bfloat16, device="cuda")
    was = out._version
    got = mx.grouped_gemm4(dev(np.array(off, np.int64)), dev(a), dev(sa), dev(b), dev(sb), elem, out=out)
    assert got is out and out._version > was
    for g in range(G):
        r = slice(off[g], off[g + 1])
        _close(got[r], *P.gemm(a[r], sa[r], b[g], sb[g], elem), K, elem, f"group {g}") if off[g] < off[g + 1] else None
    left = torch.cat([got[:off[0]], got[off[-1]:]])
    assert (left == -3.0).all()                   # rows of no group stay as they were


@pytest.mark.parametrize("elem", ["e4m3", "e2m1"])
def test_grouped_many_tiles(elem):
    """Hundreds of tiles of uneven groups."""
    rng = np.random.default_rng(3)
    sizes = rng.integers(0, 700, 16)
    sizes[3] = 0
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)
    T, N, K = int(off[-1]), 1288, 1024
    a, sa = _operand((T, K), elem, 1)
    b, sb = _operand((16, N, K), "e2m1", 2)
    got = mx.grouped_gemm4(dev(off), dev(a), dev(sa), dev(b), dev(sb), elem)
    for g in range(16):
        r = slice(off[g], off[g + 1])
        if sizes[g]:
            _close(got[r], *P.gemm(a[r], sa[r], b[g], sb[g], elem), K, elem, f"group {g}")


@pytest.mark.parametrize("elem", ELEMS)
@pytest.mark.parametrize("K", [128, 416, 1056, 1312])
def test_grouped_long_groups_of_any_length(elem, K):
    rng = np.random.default_rng(K)
    sizes = rng.integers(100, 700, 12)
    sizes[5] = 0
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)
    T, N, G = int(off[-1]) + 3, 2603, len(sizes)
    a, sa = _operand((T, K), elem, 1)
    b, sb = _operand((G, N, K), "e2m1", 2)
    out = torch.full((T, N), -3.0, dtype=torch.bfloat16, device="cuda")
    got = mx.grouped_gemm4(dev(off), dev(a), dev(sa), dev(b), dev(sb), elem, out=out)
    for g in range(G):
        r = slice(off[g], off[g + 1])
        if sizes[g]:
            _close(got[r], *P.gemm(a[r], sa[r], b[g], sb[g], elem), K, elem, f"group {g}")
    assert (got[T - 3:] == -3.0).all()


@pytest.mark.parametrize("K", [512, 544])
def test_grouped_large_with_bad_offsets_stays_in_bounds(K):
    T, N = 6000, 2600
    a, sa = _operand((T, K), "e4m3", 1)
    b, sb = _operand((3, N, K), "e2m1", 2)
    guard = torch.full((T + 300, N), -3.0, dtype=torch.bfloat16, device="cuda")
    for off in ([0, T + 900, 2, T], [-5, 3, 1 << 40, T], [T, 1, 0, T]):
        mx.grouped_gemm4(dev(np.array(off, np.int64)), dev(a), dev(sa), dev(b), dev(sb), out=guard[:T])
        assert (guard[T:] == -3.0).all()


@pytest.mark.parametrize("elem", ["e4m3", "e2m1"])
@pytest.mark.parametrize("T", [150, 700])
def test_grouped_one_group_has_most_rows(elem, T):
    """Many row tiles of one group, none of most others, more than 64 groups."""
    G, N, K = 70, 140, 288
    sizes = np.zeros(G, np.int64)
    sizes[[2, 66, 69]] = 3, T - 5, 2
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)
    a, sa = _operand((T, K), elem, 1)
    b, sb = _operand((G, N, K), "e2m1", 2)
    got = mx.grouped_gemm4(dev(off), dev(a), dev(sa), dev(b), dev(sb), elem)
    for g in (2, 66, 69):
        r = slice(off[g], off[g + 1])
        _close(got[r], *P.gemm(a[r], sa[r], b[g], sb[g], elem), K, elem, f"group {g}")


def test_grouped_more_row_tiles_than_a_grid_takes():
    """Ones times ones over 65600 tiles of 128 rows: every row is 32."""
    T = 128 * 65600
    a = torch.full((T, 32), 0x38, dtype=torch.uint8, device="cuda")
    s = torch.full((T, 1), 127, dtype=torch.uint8, device="cuda")
    b = torch.full((2, 3, 16), 0x22, dtype=torch.uint8, device="cuda")
    sb = torch.full((2, 3, 1), 127, dtype=torch.uint8, device="cuda")
    sb[1] = 128                                   # the second group's weight is 2
    off = dev(np.array([0, T - 1000, T], np.int64))
    c = mx.grouped_gemm4(off, a, s, b, sb)
    assert (c[:T - 1000] == 32).all() and (c[T - 1000:] == 64).all()


def test_not_a_number_at_the_end_of_a_row_stays_there():
    """A row whose last scale is NaN leaves the others as they were."""
    M, N, K = 3301, 3301, 416
    a, sa = _operand((M, K), "e4m3", 1)
    b, sb = _operand((N, K), "e2m1", 2)
    whole = mx.gemm4(dev(a), dev(sa), dev(b), dev(sb))
    sa[5, -1] = sb[7, -1] = 255
    got = mx.gemm4(dev(a), dev(sa), dev(b), dev(sb))
    nan = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    nan[5] = nan[:, 7] = True
    assert torch.isnan(got[nan]).all()
    assert torch.equal(got[~nan].view(torch.int16), whole[~nan].view(torch.int16))


@pytest.mark.parametrize("T", [8, 600])
def test_grouped_with_bad_offsets_stays_in_bounds(T):
    """Offsets past the rows, negative or decreasing: wrong rows, none outside."""
    a, sa = _operand((T, 512), "e4m3", 1)
    b, sb = _operand((3, 64, 512), "e2m1", 2)
    guard = torch.full((T + 64, 64), -3.0, dtype=torch.bfloat16, device="cuda")
    for off in ([0, T + 900, 2, T], [-5, 3, 1 << 40, T], [T, 1, 0, T]):
        mx.grouped_gemm4(dev(np.array(off, np.int64)), dev(a), dev(sa), dev(b), dev(sb), out=guard[:T])
        assert (guard[T:] == -3.0).all()


def test_rows_do_not_depend_on_their_neighbours():
    """A row's result is the same bits alone and in a batch of the same kernel."""
    a, sa = _operand((16, 2048), "e4m3", 1)
    b, sb = _operand((96, 2048), "e2m1", 2)
    w = dev(b), dev(sb)
    all_ = mx.gemm4(dev(a), dev(sa), *w)
    for r in (0, 7, 15):
        assert torch.equal(mx.gemm4(dev(a[r:r + 1]), dev(sa[r:r + 1]), *w)[0], all_[r])


@pytest.mark.parametrize("M", [1, 64, 700])
def test_repeats_streams_and_graphs(M):
    """The same bits on every call, on another stream and in replays of two
    graphs that were captured side by side."""
    N, K = 520, 2048
    a, sa = _operand((M, K), "e4m3", 1)
    b, sb = _operand((N, K), "e2m1", 2)
    args = dev(a), dev(sa), dev(b), dev(sb)
    off = dev(np.array([0, M // 3, M], np.int64))
    gargs = off, args[0], args[1], torch.stack([args[2]] * 2), torch.stack([args[3]] * 2)
    want, gwant = mx.gemm4(*args), mx.grouped_gemm4(*gargs)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again, gagain = mx.gemm4(*args), mx.grouped_gemm4(*gargs)
    here = mx.gemm4(*args)                        # at the same time on the current stream
    side.synchronize()
    assert torch.equal(again, want) and torch.equal(gagain, gwant) and torch.equal(here, want)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = mx.gemm4(*args), mx.grouped_gemm4(*gargs)
        graphs.append((g, outs))
    for _ in range(3):
        for g, outs in graphs:
            for t in outs:
                t.zero_()
            g.replay()
        (want.float() @ want.float().t()).sum().item()
        for g, outs in graphs:
            assert torch.equal(outs[0], want) and torch.equal(outs[1], gwant)


def test_refusals():
    a, sa = (dev(t) for t in _operand((4, 64), "e4m3", 1))
    b, sb = (dev(t) for t in _operand((8, 64), "e2m1", 2))
    with pytest.raises(ValueError):
        mx.gemm4(a, sa, b[:, :16].contiguous(), sb)
    with pytest.raises(ValueError):
        mx.gemm4(a, sa[:2], b, sb)
    with pytest.raises(ValueError):
        mx.gemm4(a, sa, b, sb, "e2m1")
    with pytest.raises(ValueError):
        mx.gemm4(a, sa, b, sb, out=torch.empty((4, 9), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        mx.gemm4(a, sa, b, sb, out=torch.empty((4, 8), dtype=torch.float32, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        mx.gemm4(a, sa, b.t().contiguous().t(), sb)
    with pytest.raises(mx.MXError, match="shares memory"):
        both = torch.zeros(1024, dtype=torch.uint8, device="cuda")
        mx.gemm4(both[:256].view(4, 64), sa, b, sb, out=both[:64].view(torch.bfloat16).view(4, 8))
    with pytest.raises(ValueError):
        mx.grouped_gemm4(torch.zeros(1, dtype=torch.int64, device="cuda"), a, sa, b[None], sb[None])
    with pytest.raises(TypeError):
        mx.grouped_gemm4(torch.zeros(2, dtype=torch.int32, device="cuda"), a, sa, b[None], sb[None])
