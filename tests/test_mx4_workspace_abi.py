"""The workspace of the product with a 4-bit weight shares no memory with what the
call reads and writes (CPU; pointers are numbers that nothing reads)."""
import pytest

import mxfp8_microscaled_precision_amd as mx

INVALID = 1
M, N, K = 64, 512, 8192
SIZES = [M * K, M * K // 32, N * K // 2, N * K // 32, 2 * M * N]     # a, sa, b, sb, c
FAR = [4096 + (i << 30) for i in range(5)]


@pytest.mark.parametrize("other", range(5))
@pytest.mark.parametrize("end", ["first", "last"])
def test_workspace_shares_no_memory(other, end):
    need = mx.mx_gemm4_workspace_size(0, M, N, K)
    assert need > 0
    # the workspace's last 16 bytes on the buffer's first, or the other way round
    ws = FAR[other] - need + 16 if end == "first" else FAR[other] + SIZES[other] - 16
    ptrs = list(FAR)
    if ws < 16:
        ptrs = [p + (1 << 29) for p in FAR]
        ws += 1 << 29
    assert mx.mx_gemm4(0, M, N, K, *ptrs, ws, need, 0) == INVALID
    assert "shares memory" in mx.mx_last_error()
