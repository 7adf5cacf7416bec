"""Refusals of routing, token movement and gradient clipping: every argument
is checked on the host before any HIP call (CPU only)."""
import ctypes

import pytest

import mxfp8_microscaled_precision_amd as mx

INVALID, SHAPE = 1, 2

# score, dtype, logits, bias, T, E, k, groups, top groups, value, renorm, scale,
# weights, experts, offsets, slots, workspace, bytes, stream
ROUTE = dict(score=0, dtype=1, logits=1, bias=0, T=4, E=64, k=8, n=1, tn=1, gv=0, renorm=1, scale=1.0,
             w=1, e=1, o=1, s=1, ws=0, nws=0, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(score=2), INVALID), (dict(score=-1), INVALID), (dict(dtype=2), INVALID),
    (dict(gv=2), INVALID), (dict(T=-1), INVALID),
    (dict(E=0), INVALID), (dict(E=513), INVALID), (dict(k=0), INVALID), (dict(k=17), INVALID),
    (dict(E=4, k=5), INVALID),
    (dict(n=0), INVALID), (dict(n=3), INVALID), (dict(n=64), INVALID),       # not a divisor; over 32
    (dict(n=8, tn=0), INVALID), (dict(n=8, tn=9), INVALID),
    (dict(n=16, tn=1, k=5), INVALID),                                        # 4 experts in one group
    (dict(T=1 << 28), SHAPE),                                                # 2^31 rows
    (dict(logits=0), INVALID), (dict(w=0), INVALID), (dict(e=0), INVALID), (dict(o=0), INVALID),
    (dict(s=0), INVALID), (dict(T=0, o=0), INVALID),
    (dict(T=1000, ws=0, nws=1 << 20), INVALID), (dict(T=1000, ws=1, nws=4), INVALID),
])
def test_route_validation(change, status):
    a = dict(ROUTE, **change)
    assert mx.mx_route(*a.values()) == status
    assert mx.mx_last_error() != ""


def test_route_workspace_size():
    assert mx.mx_route_workspace_size(0, 64) == 0
    assert mx.mx_route_workspace_size(1, 64) == 0
    assert mx.mx_route_workspace_size(16384, 64) > 0
    assert mx.mx_route_workspace_size(-1, 64) == 0
    assert mx.mx_route_workspace_size(16384, 513) == 0


@pytest.mark.parametrize("args,status", [
    ((2, 1, 1, 1, 1, 4, 8, 2, 1, 1.0, 1, 0), INVALID),
    ((0, 5, 1, 1, 1, 4, 8, 2, 1, 1.0, 1, 0), INVALID),
    ((0, 1, 1, 1, 1, -4, 8, 2, 1, 1.0, 1, 0), INVALID),
    ((0, 1, 1, 1, 1, 4, 8, 9, 1, 1.0, 1, 0), INVALID),
    ((0, 1, 1, 1, 1, 1 << 28, 8, 1, 1, 1.0, 1, 0), SHAPE),
    ((0, 1, 0, 1, 1, 4, 8, 2, 1, 1.0, 1, 0), INVALID),
    ((0, 1, 1, 0, 1, 4, 8, 2, 1, 1.0, 1, 0), INVALID),
    ((0, 1, 1, 1, 0, 4, 8, 2, 1, 1.0, 1, 0), INVALID),
    ((0, 1, 1, 1, 1, 4, 8, 2, 1, 1.0, 0, 0), INVALID),
    ((0, 1, 0, 0, 0, 0, 8, 2, 1, 1.0, 0, 0), 0),                             # no token: no-op
])
def test_route_backward_validation(args, status):
    assert mx.mx_route_backward(*args) == status


@pytest.mark.parametrize("args,status", [
    # x, T, H, k, E, offsets, slots, y, stream
    ((1, -1, 64, 2, 8, 1, 1, 1, 0), INVALID), ((1, 4, -1, 2, 8, 1, 1, 1, 0), INVALID),
    ((1, 4, 64, 0, 8, 1, 1, 1, 0), INVALID), ((1, 4, 64, 17, 64, 1, 1, 1, 0), INVALID),
    ((1, 4, 64, 2, 0, 1, 1, 1, 0), INVALID), ((1, 4, 64, 2, 513, 1, 1, 1, 0), INVALID),
    ((1, 1 << 30, 64, 2, 8, 1, 1, 1, 0), SHAPE), ((1, 1 << 26, 512, 2, 8, 1, 1, 1, 0), SHAPE),
    ((1, 4, 1 << 41, 2, 8, 1, 1, 1, 0), SHAPE),
    ((0, 4, 64, 2, 8, 1, 1, 1, 0), INVALID), ((1, 4, 64, 2, 8, 0, 1, 1, 0), INVALID),
    ((1, 4, 64, 2, 8, 1, 0, 1, 0), INVALID), ((1, 4, 64, 2, 8, 1, 1, 0, 0), INVALID),
    ((0, 0, 64, 2, 8, 0, 0, 0, 0), 0), ((0, 4, 0, 2, 8, 0, 0, 0, 0), 0),
])
def test_dispatch_validation(args, status):
    assert mx.mx_dispatch(*args) == status
    x, T, H, k, E, o, s, y, st = args
    assert mx.mx_dispatch_quant(0, x, T, H, k, E, o, s, y, y, st) == status
    # combine: y, T, H, k, slots, weights, residual, out
    if o and E in (8, 64):
        assert mx.mx_combine(x, T, H, k, s, 0, 0, y, st) == status


def test_dispatch_quant_validation():
    assert mx.mx_dispatch_quant(2, 1, 4, 64, 2, 8, 1, 1, 1, 1, 0) == INVALID
    assert mx.mx_dispatch_quant(0, 1, 4, 48, 2, 8, 1, 1, 1, 1, 0) == SHAPE
    assert mx.mx_dispatch_quant(0, 1, 4, 64, 2, 8, 1, 1, 1, 0, 0) == INVALID


@pytest.mark.parametrize("args,status", [
    # dout, y, T, H, k, E, offsets, slots, weights, dy, dweights, stream
    ((1, 1, -1, 64, 2, 8, 1, 1, 1, 1, 1, 0), INVALID),
    ((1, 1, 1 << 24, 64, 2, 8, 1, 1, 1, 1, 1, 0), SHAPE),
    ((0, 1, 4, 64, 2, 8, 1, 1, 1, 1, 1, 0), INVALID), ((1, 0, 4, 64, 2, 8, 1, 1, 1, 1, 1, 0), INVALID),
    ((1, 1, 4, 64, 2, 8, 0, 1, 1, 1, 1, 0), INVALID), ((1, 1, 4, 64, 2, 8, 1, 0, 1, 1, 1, 0), INVALID),
    ((1, 1, 4, 64, 2, 8, 1, 1, 0, 1, 1, 0), INVALID), ((1, 1, 4, 64, 2, 8, 1, 1, 1, 0, 1, 0), INVALID),
    ((1, 1, 4, 64, 2, 8, 1, 1, 1, 1, 0, 0), INVALID),
    ((0, 0, 0, 64, 2, 8, 0, 0, 0, 0, 0, 0), 0),
])
def test_combine_backward_validation(args, status):
    assert mx.mx_combine_backward(*args) == status


def _grad(ptrs, sizes, codes, max_norm=None, norm=1, ws=1, nws=1 << 20):
    n = len(ptrs)
    p, s, c = (ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*sizes), (ctypes.c_int * n)(*codes)
    if max_norm is None:
        return mx.mx_grad_norm(n, p, s, c, norm, ws, nws, 0)
    return mx.mx_grad_clip(n, p, s, c, max_norm, norm, ws, nws, 0)


@pytest.mark.parametrize("max_norm", [None, 1.0])
def test_grad_validation(max_norm):
    assert _grad([0], [4], [1], max_norm) == INVALID                  # NULL tensor
    assert _grad([64], [-4], [1], max_norm) == INVALID                # negative size
    assert _grad([64], [4], [2], max_norm) == INVALID                 # unknown type
    assert _grad([66], [4], [1], max_norm) == INVALID                 # FP32 off its alignment
    assert _grad([65], [4], [0], max_norm) == INVALID                 # BF16 off its alignment
    assert _grad([64], [1 << 41], [0], max_norm) == SHAPE
    assert _grad([64, 1 << 46], [1 << 39, 1 << 39], [1, 1], max_norm) == SHAPE
    assert _grad([64], [4], [1], max_norm, norm=0) == INVALID
    assert _grad([64], [4], [1], max_norm, ws=0) == INVALID
    assert _grad([64], [4], [1], max_norm, nws=8) == INVALID
    assert mx.mx_last_error() != ""


def test_grad_clip_validation():
    assert _grad([64], [4], [1], -1.0) == INVALID
    assert _grad([64], [4], [1], float("nan")) == INVALID
    assert _grad([64, 72], [4, 4], [1, 1], 1.0) == INVALID            # 64..80 and 72..88
    assert "share memory" in mx.mx_last_error()
    assert _grad([128, 64, 64], [4, 4, 4], [0, 0, 0], 1.0) == INVALID  # the same tensor twice


def test_grad_workspace_size():
    assert mx.mx_grad_norm_workspace_size(0) == 0
    assert mx.mx_grad_norm_workspace_size(-3) == 0
    assert mx.mx_grad_norm_workspace_size(1) > 0
    assert mx.mx_grad_norm_workspace_size(1000) > mx.mx_grad_norm_workspace_size(1)


def test_binding_refuses_cpu_tensors_and_unknown_names():
    import torch
    x = torch.zeros(4, 8)
    r = mx.Routing(torch.zeros(4, 2), torch.zeros(4, 2, dtype=torch.int32),
                   torch.zeros(9, dtype=torch.int64), torch.zeros(4, 2, dtype=torch.int32))
    b = x.to(torch.bfloat16)
    with pytest.raises(ValueError):
        mx.route(x, 2, score="tanh")
    with pytest.raises(ValueError):
        mx.route(x, 2, group_value="mean")
    with pytest.raises(ValueError):
        mx.route_backward(x, x, x, score="tanh")
    with pytest.raises(ValueError):
        mx.dispatch_quant(b, r, "int8")
    for call in (lambda: mx.route(x, 2), lambda: mx.route(x.half(), 2), lambda: mx.dispatch(b, r),
                 lambda: mx.dispatch_quant(b, r), lambda: mx.combine(b, r),
                 lambda: mx.combine_backward(b, b, r), lambda: mx.grad_norm([x]),
                 lambda: mx.grad_clip([x], 1.0), lambda: mx.grad_norm([x.half()]),
                 lambda: mx.route_backward(x, x, x)):
        with pytest.raises(TypeError):
            call()


# Sizes at which a launch grid, rounded up to whole workgroups of 256
# work-items, would hold 2^32 of them.  The last size that fits is told from
# the first that does not by what comes next: the check for NULL pointers.

@pytest.mark.parametrize("over,status", [(0, INVALID), (1, SHAPE), (2, SHAPE), (3, SHAPE)])
def test_move_grid_limit(over, status):
    T = (1 << 26) - 4 + over                                              # rows of 512: one wave a token
    assert mx.mx_dispatch(0, T, 512, 1, 8, 0, 0, 0, 0) == status
    assert mx.mx_dispatch_quant(0, 0, T, 512, 1, 8, 0, 0, 0, 0, 0) == status
    assert mx.mx_combine(0, T, 512, 1, 0, 0, 0, 0, 0) == status
    # three waves a token: 3 T <= 2^26 - 4
    assert mx.mx_dispatch(0, 22369620 + over, 1025, 1, 8, 0, 0, 0, 0) == status


@pytest.mark.parametrize("over,status", [(0, INVALID), (1, SHAPE), (15, SHAPE)])
def test_route_backward_grid_limit(over, status):
    T = (1 << 28) - 16 + over
    assert mx.mx_route_backward(0, 1, 0, 0, 0, T, 8, 1, 1, 1.0, 0, 0) == status


@pytest.mark.parametrize("over,status", [(0, INVALID), (1, SHAPE)])
def test_combine_backward_grid_limit(over, status):
    T = (1 << 24) - 1 + over                                              # a workgroup a token
    assert mx.mx_combine_backward(0, 0, T, 64, 1, 8, 0, 0, 0, 0, 0, 0) == status


@pytest.mark.parametrize("where", ["start", "end", "inside", "same"])
def test_combine_refuses_an_output_that_shares_memory(where):
    """y is read by other waves after out's rows are written, so out may not
    share memory with y, slots or weights, nor with a part of residual."""
    # T = 4, H = 64, k = 2: out and residual 512 bytes, y 1024, slots and weights 32
    far = {"y": 0x100000, "slots": 0x200000, "weights": 0x300000, "residual": 0x400000}
    size = {"y": 1024, "slots": 32, "weights": 32, "residual": 512}

    def call(out):
        return mx.mx_combine(far["y"], 4, 64, 2, far["slots"], far["weights"], far["residual"], out, 0)

    for name in far:
        lo, hi = far[name], far[name] + size[name]
        out = {"start": lo - 510, "end": hi - 2, "inside": lo + 2, "same": lo}[where]
        if name == "residual" and where == "same":
            continue                                                      # allowed, whole
        assert call(out) == INVALID, name
        assert "shares memory" in mx.mx_last_error()
