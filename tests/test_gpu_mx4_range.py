"""The 4-bit and checkpoint calls where sizes and offsets pass 32 bits: parts of
a large tensor against the same calls on those parts alone."""
import gc

import pytest
import torch

import mxfp8_microscaled_precision_amd as mx

pytestmark = pytest.mark.gpu

ONE = {"e4m3": 0x38, "e5m2": 0x3C, "e2m1": 2}


@pytest.fixture(autouse=True)
def _memory():
    gc.collect()
    torch.cuda.empty_cache()
    yield
    gc.collect()
    torch.cuda.empty_cache()


def _normal(shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)


def _codes(shape, seed, high=256):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, dtype=torch.uint8, device="cuda").random_(0, high, generator=g)


def _one_hot(rows, at, K, elem):
    """Row r of zeros but for a code 1 at column at[r]."""
    q = torch.zeros((rows, K // 2 if elem == "e2m1" else K), dtype=torch.uint8, device="cuda")
    r = torch.arange(rows, device="cuda")
    if elem == "e2m1":
        q[r, at // 2] = (ONE[elem] << (4 * (at % 2))).to(torch.uint8)
    else:
        q[r, at] = ONE[elem]
    return q, torch.full((rows, K // 32), 127, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("elem,M,N,K", [
    ("e4m3", 1, 40, 2 ** 23 - 32), ("e2m1", 1, 40, 2 ** 23 - 32), ("e5m2", 48, 130, 2 ** 23 - 32),
    ("e4m3", 200, 130, 2 ** 23 - 32), ("e2m1", 200, 130, 2 ** 23 - 32),
    # tiles of 256 rows, with whole groups of scales and without
    ("e4m3", 8192, 2048, 2 ** 23 - 512), ("e4m3", 8192, 2048, 2 ** 23 - 32), ("e2m1", 8192, 2048, 2 ** 23 - 32)])
def test_gemm4_longest_rows(elem, M, N, K):
    """One-hot rows: the weight's column at the row's ends and in between."""
    at = torch.tensor([0, 31, 32, 127, 128, 4095, K // 2, K - 129, K - 128, K - 33, K - 32, K - 1], device="cuda")
    b = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    b[:, at // 2] = _codes((N, len(at)), 1)
    sb = torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda")
    sb[:, (at // 32)] = 120 + _codes((N, len(at)), 2, 12)
    for first in (0, 5) if M == 1 else (0,):
        pos = at[(torch.arange(M, device="cuda") + first) % len(at)]
        a, sa = _one_hot(M, pos, K, elem)
        got = mx.gemm4(a, sa, b, sb, elem)
        block = b.view(N, K // 32, 16)[:, at // 32].reshape(N, -1)     # each position's block, restored
        w = mx.dequant(block, sb[:, at // 32].contiguous(), "e2m1").view(N, len(at), 32)
        w = w[:, torch.arange(len(at), device="cuda"), at % 32]
        want = w[:, (torch.arange(M, device="cuda") + first) % len(at)].t()
        assert torch.equal(got, want)


@pytest.mark.parametrize("elem", ["e4m3", "e2m1"])
@pytest.mark.parametrize("T,G,N,K", [(1030, 512, 4128, 8224), (600000, 512, 4096, 8192)])
def test_grouped_weights_and_rows_past_4_gb(T, G, N, K, elem):
    off = torch.linspace(0, T, G + 1, dtype=torch.float64, device="cuda").long()
    a, sa = _one_hot(T, (torch.arange(T, device="cuda") * 977) % K, K, elem)
    b, sb = _codes((G, N, K // 2), 3), 120 + _codes((G, N, K // 32), 4, 12)
    got = mx.grouped_gemm4(off, a, sa, b, sb, elem)
    for g in (0, 1, G // 2, G - 2, G - 1):
        r = slice(int(off[g]), int(off[g + 1]))
        assert torch.equal(got[r], mx.gemm4(a[r], sa[r], b[g], sb[g], elem))


def test_quant4_and_dequant_past_4_g_elements():
    rows, cols = 131072 + 32, 36864 + 32
    x = _normal((rows, cols), 5)
    q, s, qt, st = mx.quant4(x, "dual")
    for r in (0, 65536, rows - 64):
        wq, ws = mx.quant4(x[r:r + 64], "row")
        assert torch.equal(q[r:r + 64], wq) and torch.equal(s[r:r + 64], ws)
    rq, rs = mx.quant4(x, "row")
    assert torch.equal(rq, q) and torch.equal(rs, s)
    del rq, rs
    for c in (0, 16384 + 32, cols - 64):
        wq, ws = mx.quant4(x[:, c:c + 64].contiguous(), "col")
        assert torch.equal(qt[c:c + 64], wq) and torch.equal(st[c:c + 64], ws)
    y = mx.dequant(q, s, "e2m1")
    for r in (0, 65536, rows - 64):
        assert torch.equal(y[r:r + 64], mx.dequant(q[r:r + 64], s[r:r + 64], "e2m1"))


@pytest.mark.parametrize("grouped", [False, True])
def test_column_blocks_past_4_gb(grouped):
    rows, cols = 131072 + 32, 36864 + 32
    q, s = mx.quant(_normal((rows, cols), 6), "row")
    if grouped:
        off = torch.tensor([0, 70001, 70001, rows], device="cuda")
        qt, st = mx.requant_grouped_col(q, s, off)
    else:
        qt, st = mx.requant_col(q, s)
    for c in (0, 16384 + 32, cols - 64):
        part = q[:, c:c + 64].contiguous(), s[:, c // 32:c // 32 + 2].contiguous()
        wq, ws = mx.requant_grouped_col(*part, off) if grouped else mx.requant_col(*part)
        assert torch.equal(qt[c:c + 64], wq) and torch.equal(st[c:c + 64], ws)


def test_swiglu_over_several_launches():
    """More chunks of eight columns than one launch numbers in 32 bits."""
    T, F = 16400, 1 << 20
    x = _normal((T, 2 * F), 7)
    q, s, (cq, cs) = mx.swiglu_quant(x)
    rows = [slice(0, 2), slice(8190, 8194), slice(16380, 16387), slice(T - 2, T)]
    for r in rows:
        wq, ws, ck = mx.swiglu_quant(x[r])
        assert torch.equal(q[r], wq) and torch.equal(s[r], ws)
        assert torch.equal(cq[r], ck[0]) and torch.equal(cs[r], ck[1])
    del x, q, s
    dh = _normal((T, F), 8)
    dx = mx.swiglu_backward(dh, cq, cs)
    for r in rows:
        assert torch.equal(dx[r], mx.swiglu_backward(dh[r], cq[r], cs[r]))
    del dx
    q, s = mx.swiglu_backward_quant(dh, cq, cs)
    for r in rows:
        wq, ws = mx.swiglu_backward_quant(dh[r], cq[r], cs[r])
        assert torch.equal(q[r], wq) and torch.equal(s[r], ws)
