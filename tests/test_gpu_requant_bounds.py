"""Column blocks from row blocks with offsets that are wrong: what is read and
what is written."""
import numpy as np
import pytest
import torch

import mxfp8_microscaled_precision_amd as mx
from parity import dev

pytestmark = pytest.mark.gpu

PAD = 4096


def _within(data, fill):
    """A copy of data with PAD bytes of `fill` on either side: (all, view)."""
    room = torch.full((data.numel() + 2 * PAD,), fill, dtype=torch.uint8, device="cuda")
    view = room[PAD:PAD + data.numel()].view(data.shape)
    view.copy_(data)
    return room, view


def _call(q, s, off, prefill):
    T, C = q.shape
    G = off.numel() - 1
    cap = mx.grouped_col_capacity(T, G)
    room_q, qt = _within(torch.full((C, cap), prefill, dtype=torch.uint8, device="cuda"), 0x3C)
    room_s, st = _within(torch.full((C, cap // 32), prefill, dtype=torch.uint8, device="cuda"), 0x3C)
    status = mx.mx_requant_grouped_col(0, 0, q.data_ptr(), s.data_ptr(), T, C, G, off.data_ptr(), qt.data_ptr(),
                                       st.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert status == 0
    for room in (room_q, room_s):
        assert (room[:PAD] == 0x3C).all() and (room[-PAD:] == 0x3C).all()
    return qt, st


@pytest.mark.parametrize("T,C", [(96, 64), (1000, 416)])
def test_bad_offsets_read_rows_of_the_source_and_write_every_block(T, C):
    """NaN codes and scales stand on either side of the source, other bytes on
    either side of the result.  Two calls over different old contents agree, so
    each byte is written; no scale is NaN, so no byte beside the source is read."""
    rng = np.random.default_rng(T)
    x = torch.from_numpy(rng.standard_normal((T, C))).to(torch.bfloat16).cuda()
    q, s = (_within(t, fill)[1] for t, fill in zip(mx.quant(x, "row"), (0x7F, 0xFF)))
    top = int(mx.requant_grouped_col(q, s, dev(np.array([0, T], np.int64)))[1].max())
    offsets = [[0, 5 * T, T], [-40, 30, T], [0, T - 6, 20, T], [7, 7, 7, 1 << 60], [T, 0, T, 0, T], [-(1 << 60), T + 1],
               [3 * T, 2 * T], [1 << 60, -(1 << 60), 5]]
    for _ in range(4):
        offsets.append(rng.integers(-T, 2 * T, 70).tolist())
    for off in offsets:
        off = dev(np.array(off, np.int64))
        one, two = _call(q, s, off, 0x11), _call(q, s, off, 0xEE)
        assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1]), off
        assert int(one[1].max()) <= top and not ((one[0] & 0x7F) == 0x7F).any(), off
