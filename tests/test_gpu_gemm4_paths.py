"""Products with 4-bit weights on the GPU, by the path that the sizes, offsets
and addresses select: exact operands, or the same bits from two calls."""
import numpy as np
import pytest
import torch

import mxfp8_microscaled_precision_amd as mx
import plain_mx4 as P
from parity import dev

pytestmark = pytest.mark.gpu

ELEMS = ["e4m3", "e5m2", "e2m1"]


def _operand(shape, elem, seed):
    rng = np.random.default_rng(seed)
    return P.quant_rows(rng.standard_normal(shape) * np.exp(rng.standard_normal(shape[:-1] + (1,))), elem)


def _at(t, shift):
    """A copy of t that begins `shift` bytes past a 256-byte boundary."""
    room = torch.empty(t.numel() + 256, dtype=torch.uint8, device="cuda")
    first = -room.data_ptr() % 256 + shift
    view = room[first:first + t.numel()].view(t.shape)
    assert view.data_ptr() % 16 == shift and view.is_contiguous()
    return view.copy_(t)


@pytest.mark.parametrize("shift_a,shift_b", [(1, 0), (0, 2), (4, 4), (8, 15), (13, 3)])
@pytest.mark.parametrize("elem", ELEMS)
@pytest.mark.parametrize("M,N,K", [(3304, 3304, 1024), (300, 520, 1024), (5, 70, 2048), (40, 33, 64)])
def test_scales_at_any_address(M, N, K, elem, shift_a, shift_b):
    """Scales need no alignment: the bits are those of aligned ones."""
    a, sa = (dev(t) for t in _operand((M, K), elem, 1))
    b, sb = (dev(t) for t in _operand((N, K), "e2m1", 2))
    want = mx.gemm4(a, _at(sa, 0), b, _at(sb, 0), elem)
    got = mx.gemm4(a, _at(sa, shift_a), b, _at(sb, shift_b), elem)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("shift_a,shift_b", [(1, 0), (0, 2), (4, 8), (13, 3)])
@pytest.mark.parametrize("elem", ELEMS)
@pytest.mark.parametrize("rows,N,K", [(400, 2600, 1024), (40, 264, 512), (5, 130, 512)])
def test_grouped_scales_at_any_address(rows, N, K, elem, shift_a, shift_b):
    sizes = np.random.default_rng(rows).integers(rows // 2, 2 * rows, 12)
    sizes[4] = 0
    off = dev(np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64))
    a, sa = (dev(t) for t in _operand((int(sizes.sum()), K), elem, 1))
    b, sb = (dev(t) for t in _operand((12, N, K), "e2m1", 2))
    want = mx.grouped_gemm4(off, a, _at(sa, 0), b, _at(sb, 0), elem)
    got = mx.grouped_gemm4(off, a, _at(sa, shift_a), b, _at(sb, shift_b), elem)
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("elem", ["e4m3", "e2m1"])
@pytest.mark.parametrize("T,G,N,K", [(40, 5, 70, 96), (150, 70, 140, 288), (1500, 12, 140, 288), (1500, 135, 40, 288),
                                     (6000, 9, 2600, 512)])
def test_bad_offsets_count_as_their_running_maximum(T, G, N, K, elem):
    """Offsets that fall, or lie outside [0, T], name the rows that their running
    maximum within [0, T] names, in every form: each row once."""
    rng = np.random.default_rng(T + G)
    a, sa = (dev(t) for t in _operand((T, K), elem, 1))
    b, sb = (dev(t) for t in _operand((G, N, K), "e2m1", 2))
    for trial in range(6):
        off = np.sort(rng.integers(0, T + 1, G + 1))
        at = rng.integers(0, G + 1, 1 + G // 8)
        off[at] = rng.integers(-T, 2 * T, len(at)) if trial < 4 else rng.choice([0, T, -1 << 60, 1 << 60], len(at))
        if trial == 5:
            off[::2] = 0                          # every group falls back to the first row
        good = np.maximum.accumulate(np.clip(off, 0, T))
        want, got = (torch.full((T, N), -3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        mx.grouped_gemm4(dev(good), a, sa, b, sb, elem, out=want)
        mx.grouped_gemm4(dev(off), a, sa, b, sb, elem, out=got)
        assert torch.equal(got.view(torch.int16), want.view(torch.int16)), trial
        assert (got[good[-1]:] == -3.0).all() and (got[:good[0]] == -3.0).all()


ONE = {"e4m3": 0x38, "e5m2": 0x3C, "e2m1": 2}


def _signs(shape, elem, rng):
    """Codes of 1 and -1 with scales 1/4 to 4: (payload, scales, values).  A sum
    of their products is a multiple of 1/16 below 2^20, exact in FP32 in any
    order; eight neighbouring products have one scale, or two 2^8 apart at most,
    and lose no bit to the matrix instruction's alignment."""
    codes = np.where(rng.random(shape) < 0.5, ONE[elem] | (8 if elem == "e2m1" else 128), ONE[elem]).astype(np.uint8)
    s = rng.integers(125, 130, shape[:-1] + (shape[-1] // 32,), dtype=np.uint8)
    q = P.pack(codes) if elem == "e2m1" else codes
    return q, s, P.values(q, s, elem)


# one to 128 rows whose contraction is split: whole steps and not, whole dwords
# of scales and not, columns of every remainder by four
SPLIT = [(1, 8, 18432), (1, 33, 8224), (1, 512, 12288), (3, 7, 12320), (5, 40, 32768), (5, 130, 8192), (32, 34, 8288),
         (32, 40, 8192), (40, 129, 8224), (64, 70, 18432), (64, 131, 8256), (100, 33, 8224), (128, 64, 4096),
         (200, 66, 4128)]


@pytest.mark.parametrize("M,N,K", SPLIT)
@pytest.mark.parametrize("elem", ELEMS)
def test_split_contraction_is_exact(M, N, K, elem):
    """Sums of signed powers of two, in which no step of 128 elements can be lost
    or counted twice without a result that differs."""
    assert mx.mx_gemm4_workspace_size(mx.OPERAND_ELEMS[elem], M, N, K) > 0
    rng = np.random.default_rng(M + N + K)
    a, sa, x = _signs((M, K), elem, rng)
    b, sb, y = _signs((N, K), "e2m1", rng)
    ref = x @ y.T
    want = P.bf16_round(ref)
    for k in range(0, K, 128):
        part = x[:, k:k + 128] @ y[:, k:k + 128].T
        assert (P.bf16_round(ref - part) != want).any() and (P.bf16_round(ref + part) != want).any()
    got = mx.gemm4(dev(a), dev(sa), dev(b), dev(sb), elem).double().cpu().numpy()
    np.testing.assert_array_equal(got, want)


@pytest.mark.parametrize("M", [1, 32, 64, 128])
@pytest.mark.parametrize("K", [8192, 8224])
@pytest.mark.parametrize("elem", ELEMS)
def test_split_contraction_takes_every_step_once(M, K, elem):
    """One code 1 a row, beside every edge of a step: the weight's column."""
    N = 33
    assert mx.mx_gemm4_workspace_size(mx.OPERAND_ELEMS[elem], M, N, K) > 0
    b, sb = _operand((N, K), "e2m1", 5)
    w = P.values(b, sb, "e2m1")
    at = np.unique(np.clip(np.concatenate([np.arange(0, K + 1, 256) + d for d in (-1, 0)]), 0, K - 1))
    if M == 1:
        at = at[::7]
    for first in range(0, len(at), M):
        rows = at[first:first + M]
        codes = np.zeros((M, K), np.uint8)
        codes[np.arange(len(rows)), rows] = ONE[elem]
        a = P.pack(codes) if elem == "e2m1" else codes
        sa = np.full((M, K // 32), 127, np.uint8)
        got = mx.gemm4(dev(a), dev(sa), dev(b), dev(sb), elem).double().cpu().numpy()
        np.testing.assert_array_equal(got[:len(rows)], w[:, rows].T)


@pytest.mark.parametrize("elem", ELEMS)
@pytest.mark.parametrize("M,N,K", [(3304, 3304, 2560), (3301, 3303, 2080)])
def test_large_tiles_over_many_scale_groups(M, N, K, elem):
    """More K than two buffers of scales hold, each block with scales of its own."""
    rng = np.random.default_rng(K)
    a, sa, x = _signs((M, K), elem, rng)
    b, sb, y = _signs((N, K), "e2m1", rng)
    got = mx.gemm4(dev(a), dev(sa), dev(b), dev(sb), elem).double().cpu().numpy()
    np.testing.assert_array_equal(got, P.bf16_round(x @ y.T))


@pytest.mark.parametrize("elem", ELEMS)
@pytest.mark.parametrize("N,K", [(2600, 2560), (2603, 2080)])
def test_grouped_large_tiles_over_many_scale_groups(N, K, elem):
    rng = np.random.default_rng(K)
    sizes = rng.integers(200, 700, 12)
    off = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int64)
    a, sa, x = _signs((int(off[-1]), K), elem, rng)
    b, sb, y = _signs((12, N, K), "e2m1", rng)
    got = mx.grouped_gemm4(dev(off), dev(a), dev(sa), dev(b), dev(sb), elem).double().cpu().numpy()
    for g in range(12):
        r = slice(off[g], off[g + 1])
        np.testing.assert_array_equal(got[r], P.bf16_round(x[r] @ y[g].T))


@pytest.mark.parametrize("elem", ["e4m3", "e2m1"])
@pytest.mark.parametrize("T,G,N,K", [(40, 5, 140, 288), (1500, 70, 140, 288), (6000, 9, 2600, 512)])
def test_grouped_graph_reads_the_offsets_of_each_replay(T, G, N, K, elem):
    rng = np.random.default_rng(T)
    a, sa = (dev(t) for t in _signs((T, K), elem, rng)[:2])
    b, sb = (dev(t) for t in _signs((G, N, K), "e2m1", rng)[:2])
    off = torch.zeros(G + 1, dtype=torch.int64, device="cuda")
    out = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    mx.grouped_gemm4(off, a, sa, b, sb, elem, out=out)
    with torch.cuda.graph(graph):
        mx.grouped_gemm4(off, a, sa, b, sb, elem, out=out)
    for top in (T, T // 2, 0, T):
        off.copy_(dev(np.sort(rng.integers(0, top + 1, G + 1))))
        out.fill_(-3.0)
        graph.replay()
        want = torch.full_like(out, -3.0)
        mx.grouped_gemm4(off, a, sa, b, sb, elem, out=want)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))
        for g in range(G):
            r = slice(int(off[g]), int(off[g + 1]))
            assert torch.equal(out[r], mx.gemm4(a[r], sa[r], b[g], sb[g], elem))     # exact in any order
        assert (out[int(off[G]):] == -3.0).all() and (out[:int(off[0])] == -3.0).all()


def test_grouped_without_a_contraction_writes_zeros():
    u8 = dict(dtype=torch.uint8, device="cuda")
    off = dev(np.array([1, 3, 3, 6], np.int64))
    out = torch.full((8, 40), -3.0, dtype=torch.bfloat16, device="cuda")
    mx.grouped_gemm4(off, torch.empty((8, 0), **u8), torch.empty((8, 0), **u8), torch.empty((3, 40, 0), **u8),
                     torch.empty((3, 40, 0), **u8), out=out)
    assert not out[1:6].any() and (out[0] == -3.0).all() and (out[6:] == -3.0).all()
