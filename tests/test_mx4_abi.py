"""Refusals of the calls for 4-bit weights and 8-bit checkpoints, before any
device work (CPU; pointers are numbers that nothing reads)."""
import pytest
import torch

import mxfp8_microscaled_precision_amd as mx

INVALID, SHAPE = 1, 2
P = 4096            # an aligned address
BIG = 1 << 62


@pytest.mark.parametrize("args,want", [
    ((3, P, 1, 32, 32, P, P, P, P, 0), INVALID),          # no 32x32 tiles in 4 bits
    ((-1, P, 1, 32, 32, P, P, P, P, 0), INVALID),
    ((0, P, -1, 32, 32, P, P, 0, 0, 0), INVALID), ((0, P, 65536, 32, 32, P, P, 0, 0, 0), INVALID),
    ((0, P, 1, -32, 32, P, P, 0, 0, 0), INVALID), ((0, P, 1, BIG, 32, P, P, 0, 0, 0), INVALID),
    ((0, P, 1, 4, 40, P, P, 0, 0, 0), SHAPE), ((1, P, 1, 33, 32, 0, 0, P, P, 0), SHAPE),
    ((2, P, 1, 32, 40, P, P, P, P, 0), SHAPE), ((1, P, 1, 32, 1 << 23, 0, 0, P, P, 0), SHAPE),
    ((1, P, 1, 1 << 31, 32, 0, 0, P, P, 0), SHAPE),
    ((0, 0, 1, 4, 32, P, P, 0, 0, 0), INVALID), ((0, P, 1, 4, 32, 0, P, 0, 0, 0), INVALID),
    ((1, P, 1, 32, 32, P, P, P, 0, 0), INVALID), ((2, P, 1, 32, 32, P, 0, P, P, 0), INVALID),
    ((0, P + 8, 1, 4, 32, P, P, 0, 0, 0), INVALID), ((0, P, 1, 4, 32, P + 1, P, 0, 0, 0), INVALID),
    ((1, P, 1, 32, 32, 0, 0, P + 4, P, 0), INVALID),
    ((0, 0, 0, 4, 32, 0, 0, 0, 0, 0), 0), ((0, 0, 1, 0, 32, 0, 0, 0, 0, 0), 0), ((2, 0, 1, 32, 0, 0, 0, 0, 0, 0), 0),
])
def test_quant4(args, want):
    assert mx.mx_quant4(*args) == want


@pytest.mark.parametrize("args,want", [
    ((2, P, P, 4, 32, P, 0), INVALID), ((5, P, P, 4, 32, P, 0), INVALID),
    ((0, P, P, -4, 32, P, 0), INVALID), ((0, P, P, BIG, 32, P, 0), INVALID),
    ((4, P, P, 4, 48, P, 0), SHAPE),
    ((4, 0, P, 4, 32, P, 0), INVALID), ((4, P, 0, 4, 32, P, 0), INVALID), ((4, P, P, 4, 32, 0, 0), INVALID),
    ((4, P + 4, P, 4, 32, P, 0), INVALID), ((4, P, P, 4, 32, P + 2, 0), INVALID),
    ((4, 0, 0, 0, 32, 0, 0), 0), ((1, 0, 0, 4, 0, 0, 0), 0),
])
def test_dequant(args, want):
    assert mx.mx_dequant(*args) == want


FAR = [P + (i << 30) for i in range(6)]   # operands well apart


@pytest.mark.parametrize("sizes,want", [
    ((2, 4, 4, 32), INVALID), ((3, 4, 4, 32), INVALID), ((5, 4, 4, 32), INVALID), ((-1, 4, 4, 32), INVALID),
    ((0, -4, 4, 32), INVALID), ((0, 4, -4, 32), INVALID), ((0, 4, 4, -32), INVALID), ((0, BIG, 64, 32), INVALID),
    ((4, 4, 4, 48), SHAPE), ((0, 4, 4, 1 << 23), SHAPE), ((0, 4, 1 << 28, 32), SHAPE),
    ((0, 1 << 24, 1 << 24, 32), SHAPE),
    ((0, 0, 4, 32), 0), ((4, 4, 0, 32), 0),
])
def test_gemm4_sizes(sizes, want):
    a, sa, b, sb, c, _ = FAR
    assert mx.mx_gemm4(*sizes, a, sa, b, sb, c, 0, 0, 0) == want


@pytest.mark.parametrize("missing", range(5))
def test_gemm4_pointers(missing):
    ptrs = FAR[:5]
    ptrs[missing] = 0
    assert mx.mx_gemm4(0, 4, 4, 32, *ptrs, 0, 0, 0) == INVALID
    assert mx.mx_grouped_gemm4(0, 2, P, 4, 4, 32, *ptrs, 0) == INVALID
    if missing in (0, 2, 4):
        ptrs[missing] = FAR[missing] + 8
        assert mx.mx_gemm4(0, 4, 4, 32, *ptrs, 0, 0, 0) == INVALID
        assert "aligned" in mx.mx_last_error()


@pytest.mark.parametrize("other", range(4))
def test_gemm4_result_shares_no_memory(other):
    ptrs = FAR[:5]
    ptrs[4] = ptrs[other]
    assert mx.mx_gemm4(4, 4, 4, 32, *ptrs, 0, 0, 0) == INVALID
    assert "shares memory" in mx.mx_last_error()
    assert mx.mx_grouped_gemm4(4, 2, P, 4, 4, 32, *ptrs, 0) == INVALID


def test_gemm4_workspace():
    size = mx.mx_gemm4_workspace_size(0, 64, 512, 8192)
    assert size > 0 and mx.mx_gemm4_workspace_size(0, 1 << 15, 1 << 14, 8192) == 0
    ptrs = FAR[:5]
    assert mx.mx_gemm4(0, 64, 512, 8192, *ptrs, FAR[5], size - 1, 0) == INVALID
    assert mx.mx_gemm4(0, 64, 512, 8192, *ptrs, 0, size, 0) == INVALID
    assert mx.mx_gemm4(0, 64, 512, 8192, *ptrs, FAR[5] + 8, size, 0) == INVALID
    assert "aligned" in mx.mx_last_error()
    for bad in ((2, 64, 512, 8192), (0, -1, 512, 8192), (0, 64, 0, 8192), (0, 64, 512, 8200), (0, 64, 1 << 28, 32)):
        assert mx.mx_gemm4_workspace_size(*bad) == 0


@pytest.mark.parametrize("sizes,want", [
    ((0, 0, P, 4, 4, 32), INVALID), ((0, 513, P, 4, 4, 32), INVALID), ((2, 2, P, 4, 4, 32), INVALID),
    ((0, 2, P, -4, 4, 32), INVALID), ((0, 2, P, 4, 4, 40), SHAPE), ((0, 2, P, 4, 4, 1 << 23), SHAPE),
    ((0, 2, P, 4, 1 << 28, 32), SHAPE), ((0, 2, 0, 4, 4, 32), INVALID),
    ((0, 2, 0, 0, 4, 32), 0), ((0, 2, 0, 4, 0, 32), 0),
])
def test_grouped_gemm4_sizes(sizes, want):
    a, sa, b, sb, c, _ = FAR
    assert mx.mx_grouped_gemm4(*sizes, a, sa, b, sb, c, 0) == want


@pytest.mark.parametrize("args,want", [
    ((4, 0, P, 4, 32, P, P, P, P, 0), INVALID), ((0, 4, P, 4, 32, P, P, P, P, 0), INVALID),
    ((0, 0, P, -4, 32, P, P, P, P, 0), INVALID), ((0, 0, P, 4, -32, P, P, P, P, 0), INVALID),
    ((0, 0, P, 4, 40, P, P, P, P, 0), SHAPE), ((0, 0, P, 1, 1 << 33, P, P, P, P, 0), SHAPE),
    ((0, 0, P, BIG, 32, P, P, P, P, 0), INVALID),
    ((0, 0, 0, 4, 32, P, P, P, P, 0), INVALID), ((0, 0, P, 4, 32, 0, P, P, P, 0), INVALID),
    ((0, 0, P, 4, 32, P, 0, P, P, 0), INVALID), ((0, 0, P, 4, 32, P, P, P, 0, 0), INVALID),
    ((0, 0, P, 4, 32, P, P, 0, P, 0), INVALID), ((0, 0, P + 8, 4, 32, P, P, P, P, 0), INVALID),
    ((0, 0, P, 4, 32, P + 8, P, P, P, 0), INVALID), ((0, 0, P, 4, 32, P, P, P + 8, P, 0), INVALID),
    ((0, 0, 0, 0, 32, 0, 0, 0, 0, 0), 0), ((1, 1, 0, 4, 0, 0, 0, 0, 0, 0), 0),
])
def test_swiglu_quant(args, want):
    assert mx.mx_swiglu_quant(*args) == want


@pytest.mark.parametrize("args,want", [
    ((4, P, P, P, 4, 32, P, 0), INVALID), ((0, P, P, P, -1, 32, P, 0), INVALID), ((0, P, P, P, 4, 16, P, 0), SHAPE),
    ((0, 0, P, P, 4, 32, P, 0), INVALID), ((0, P, 0, P, 4, 32, P, 0), INVALID), ((0, P, P, 0, 4, 32, P, 0), INVALID),
    ((0, P, P, P, 4, 32, 0, 0), INVALID), ((0, P + 2, P, P, 4, 32, P, 0), INVALID),
    ((0, P, P + 2, P, 4, 32, P, 0), INVALID), ((0, P, P, P, 4, 32, P + 2, 0), INVALID),
    ((1, 0, 0, 0, 0, 32, 0, 0), 0), ((1, 0, 0, 0, 4, 0, 0, 0), 0),
])
def test_swiglu_backward(args, want):
    assert mx.mx_swiglu_backward(*args) == want


@pytest.mark.parametrize("args,want", [
    ((4, 0, P, P, P, 4, 32, P, P, 0), INVALID), ((0, 4, P, P, P, 4, 32, P, P, 0), INVALID),
    ((0, 0, P, P, P, 4, 32, 0, P, 0), INVALID), ((0, 0, P, P, P, 4, 32, P, 0, 0), INVALID),
    ((0, 0, P, P, P, 4, 33, P, P, 0), SHAPE), ((0, 1, 0, 0, 0, 0, 32, 0, 0, 0), 0),
])
def test_swiglu_backward_quant(args, want):
    assert mx.mx_swiglu_backward_quant(*args) == want


@pytest.mark.parametrize("args,want", [
    ((4, 0, P, P, 32, 32, P, P, 0), INVALID), ((0, 4, P, P, 32, 32, P, P, 0), INVALID),
    ((0, 0, P, P, -32, 32, P, P, 0), INVALID), ((0, 0, P, P, 40, 32, P, P, 0), SHAPE),
    ((0, 0, P, P, 32, 40, P, P, 0), SHAPE), ((0, 0, P, P, 1 << 30, 32, P, P, 0), SHAPE),
    ((0, 0, P, P, 32, 1 << 24, P, P, 0), SHAPE),
    ((0, 0, 0, P, 32, 32, P, P, 0), INVALID), ((0, 0, P, 0, 32, 32, P, P, 0), INVALID),
    ((0, 0, P, P, 32, 32, 0, P, 0), INVALID), ((0, 0, P, P, 32, 32, P, 0, 0), INVALID),
    ((0, 0, P + 8, P, 32, 32, P, P, 0), INVALID), ((0, 0, P, P, 32, 32, P + 8, P, 0), INVALID),
    ((0, 0, 0, 0, 0, 32, 0, 0, 0), 0), ((0, 0, 0, 0, 32, 0, 0, 0, 0), 0),
])
def test_requant_col(args, want):
    assert mx.mx_requant_col(*args) == want


@pytest.mark.parametrize("args,want", [
    ((4, 0, P, P, 8, 32, 2, P, P, P, 0), INVALID), ((0, 2, P, P, 8, 32, 2, P, P, P, 0), INVALID),
    ((0, 0, P, P, 8, 32, 0, P, P, P, 0), INVALID), ((0, 0, P, P, 8, 32, 513, P, P, P, 0), INVALID),
    ((0, 0, P, P, -8, 32, 2, P, P, P, 0), INVALID), ((0, 0, P, P, 8, 40, 2, P, P, P, 0), SHAPE),
    ((0, 0, P, P, 1 << 23, 32, 2, P, P, P, 0), SHAPE),
    ((0, 0, 0, P, 8, 32, 2, P, P, P, 0), INVALID), ((0, 0, P, P, 8, 32, 2, 0, P, P, 0), INVALID),
    ((0, 0, P, P, 8, 32, 2, P, 0, P, 0), INVALID), ((0, 0, P, P, 8, 32, 2, P, P, 0, 0), INVALID),
    ((0, 0, 0, 0, 0, 0, 2, 0, 0, 0, 0), 0),
])
def test_requant_grouped_col(args, want):
    assert mx.mx_requant_grouped_col(*args) == want


def test_earlier_calls_refuse_four_bits():
    assert mx.mx_quant_elem(0, 4, P, 4, 32, P, P, 0, 0, 0) == INVALID
    assert mx.mx_gemm_elem(0, 0, 4, 4, 4, 4, 32, P, P, P, P, P, 0) == INVALID
    assert mx.mx_grouped_gemm_elem(4, 4, 1, P, 4, 4, 32, P, P, P, P, P, 0, 0, 0) == INVALID
    assert mx.mx_dispatch_quant(4, P, 4, 64, 2, 8, P, P, P, P, 0) == INVALID


def test_binding_refuses_names_and_host_tensors():
    x, u = torch.zeros((32, 64), dtype=torch.bfloat16), torch.zeros((32, 64), dtype=torch.uint8)
    for call in (lambda: mx.quant4(x, "32x32"), lambda: mx.quant4(x, "rows"), lambda: mx.dequant(u, u, "e3m2"),
                 lambda: mx.gemm4(u, u, u, u, "fp4"), lambda: mx.grouped_gemm4(u, u, u, u, u, "bf16"),
                 lambda: mx.swiglu_quant(x, "e2m1"), lambda: mx.swiglu_quant(x, checkpoint_elem="e2m1"),
                 lambda: mx.swiglu_backward(x, u, u, "e2m1"), lambda: mx.swiglu_backward_quant(x, u, u, "e2m1"),
                 lambda: mx.requant_col(u, u, "e2m1"), lambda: mx.requant_grouped_col(u, u, u, "e4m3", "e2m1"),
                 lambda: mx.quant(x, "row", "e2m1"), lambda: mx.gemm(u, u, u, u, b_elem="e2m1")):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mx.quant4(x), lambda: mx.dequant(u, u), lambda: mx.gemm4(u, u, u, u),
                 lambda: mx.grouped_gemm4(u, u, u, u, u), lambda: mx.swiglu_quant(x),
                 lambda: mx.swiglu_backward(x, u, u), lambda: mx.swiglu_backward_quant(x, u, u),
                 lambda: mx.requant_col(u, u), lambda: mx.requant_grouped_col(u, u, u)):
        with pytest.raises(TypeError):
            call()
