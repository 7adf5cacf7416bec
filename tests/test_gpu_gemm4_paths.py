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
