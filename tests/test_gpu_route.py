"""Routing on the GPU against the plain 64-bit implementation: the choice,
offsets and slots exactly, weights and gradients within derived bounds."""
import numpy as np
import pytest
import torch

import mxfp8_microscaled_precision_amd as mx
import plain_moe as P
from parity import dev, host, say

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24                      # half a step of FP32, relative


def _logits(T, E, seed, dtype="float32", mask=0.0, coarse=False):
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(T, E)) * 1.5 + rng.normal(size=(1, E)) * 0.5
    if coarse:                        # few distinct values: ties everywhere
        x = np.round(x) + 0.25
    x[rng.random((T, E)) < mask] = -np.inf
    return torch.from_numpy(x.astype(np.float32)).to(getattr(torch, dtype))


def _weight_tol(x, w, E):
    """Each exponential takes a difference rounded to half a step (an error of
    |difference| half steps of the result) and is off by a step itself; sums
    of positive terms, quotients and the scale add their roundings."""
    with np.errstate(all="ignore"):
        r = np.where(np.isfinite(x), np.abs(x), 0.0).max(1, keepdims=True)
    return (24 + E / 16 + 8 * r) * EPS * np.abs(w) + 1e-37


def _check(x, k, score="softmax", bias=None, n_groups=1, top_groups=1, group_value="top2",
           renormalize=True, scale=1.0, r=None):
    x64 = x.double().numpy()
    b64 = None if bias is None else bias.double().numpy()
    if r is None:
        r = mx.route(x.cuda(), k, score, None if bias is None else bias.cuda(), n_groups=n_groups,
                     top_groups=top_groups, group_value=group_value, renormalize=renormalize,
                     scale=scale)
    T, E = x.shape
    e = P.choose(x64, k, score, b64, n_groups, top_groups, group_value)
    np.testing.assert_array_equal(host(r.experts), e)
    off, slots = P.layout(e, E)
    np.testing.assert_array_equal(host(r.offsets), off)
    np.testing.assert_array_equal(host(r.slots), slots)
    w = P.weights(x64, e, score, renormalize, scale)
    got = host(r.weights).astype(np.float64)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(w))
    fine = ~np.isnan(w)
    tol = _weight_tol(x64, np.where(fine, w, 0.0), E)
    assert (np.abs(np.where(fine, got - w, 0.0)) <= tol).all()
    return r


@pytest.mark.parametrize("T,E,k", [
    (1, 1, 1), (1, 64, 8), (2, 3, 3), (5, 8, 2), (63, 60, 6), (64, 64, 8), (65, 65, 9), (129, 127, 4),
    (300, 128, 16), (257, 250, 6), (1000, 256, 8), (513, 257, 1), (400, 512, 12), (333, 511, 16),
    (16385, 64, 8), (40000, 16, 4),
])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_sizes(T, E, k, dtype):
    x = _logits(T, E, T + E, dtype)
    _check(x, k, "softmax")
    _check(x, k, "sigmoid", renormalize=False, scale=2.5)
    _check(x, k, "softmax", renormalize=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,n,tn", [
    (1, 64, 8, 8, 4), (70, 64, 6, 8, 3), (100, 256, 8, 8, 4), (65, 60, 5, 6, 2), (200, 512, 16, 32, 7),
    (90, 32, 4, 32, 5), (33, 96, 8, 2, 1), (1025, 160, 6, 8, 3),
])
@pytest.mark.parametrize("value", ["top2", "max"])
def test_groups(score, T, E, k, n, tn, value):
    x = _logits(T, E, 7 * T + E, mask=0.05)
    rng = np.random.default_rng(E)
    bias = torch.from_numpy((0.1 * rng.normal(size=E)).astype(np.float32))
    for b in (None, bias):
        _check(x, k, score, b, n, tn, value, scale=2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_bias_decides_and_weights_do_not_see_it(score):
    x = _logits(200, 100, 5)
    bias = torch.from_numpy(np.random.default_rng(1).normal(size=100).astype(np.float32) * 3)
    _check(x, 7, score, bias)
    _check(x, 7, score, bias, renormalize=False)
    bias[3] = -float("inf")           # an expert taken out
    r = _check(x, 7, score, bias)
    assert not (host(r.experts) == 3).any()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups", [(64, 8, 1), (256, 8, 8), (60, 16, 4), (512, 8, 1)])
def test_values_closer_than_32_bits(score, E, k, groups):
    """Biases that bring all choice values within a few 2^-25 of each other:
    only 64-bit values order them."""
    rng = np.random.default_rng(E)
    x = torch.from_numpy(rng.normal(size=E).astype(np.float32)).repeat(40, 1)
    s = P.scores(x[:1].double().numpy(), score)[0]
    bias = torch.from_numpy((0.75 - s).astype(np.float32))
    perm = torch.from_numpy(np.stack([rng.permutation(E) for _ in range(40)]))
    _check(x, k, score, bias, groups, max(1, groups // 2))
    # rows of which only some are close, among ordinary ones
    y = torch.gather(x, 1, perm)
    y[::3] = x[::3]
    _check(y, k, score, bias, groups, max(1, groups // 2))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("bias", [False, True])
def test_ties_go_to_the_lowest_index(dtype, bias):
    x = _logits(500, 256, 3, dtype, mask=0.1, coarse=True)
    b = torch.zeros(256) if bias else None
    for score in ("softmax", "sigmoid"):
        _check(x, 8, score, b)
        _check(x, 8, score, b, 8, 4, "max")
    x = torch.zeros(70, 64, dtype=x.dtype)
    x[::2] = -0.0
    r = _check(x, 8, "softmax", b[:64] if bias else None, 8, 4)
    assert (host(r.experts) == np.arange(8)).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("groups", [1, 4])
def test_masked_rows_infinities_and_nan(score, bias, groups):
    x = _logits(80, 64, 9, mask=0.3)
    inf, nan = float("inf"), float("nan")
    x[0] = -inf                       # a padding token
    x[1, 1:] = -inf                   # one expert left
    x[2, :4] = inf                    # several infinite logits
    x[3, 7] = nan
    x[4] = nan
    x[5] = -inf
    x[5, 63] = nan                    # masked but for a NaN
    x[6] = torch.finfo(torch.float32).min
    x[7] = -inf
    x[7, 20:23] = torch.finfo(torch.float32).min   # a mask of the type's lowest value
    x[8] = -300.0                     # every sigmoid underflows
    x[8, 5] = -299.0
    x[9, 9] = inf
    x[10] = torch.finfo(torch.float32).max
    b = torch.from_numpy(np.random.default_rng(1).normal(size=64).astype(np.float32)) if bias else None
    for renormalize in (True, False):
        _check(x, 8, score, b, groups, max(1, groups // 2), "max", renormalize)
        if groups > 1:
            _check(x, 8, score, b, groups, 2, "top2", renormalize)


def test_all_tokens_masked_and_no_token():
    x = torch.full((1000, 64), -float("inf"))
    r = _check(x, 8)
    assert host(r.offsets).sum() == 0 and (host(r.slots) == -1).all() and (host(r.weights) == 0).all()
    r = mx.route(torch.empty((0, 64), device="cuda"), 8)
    assert r.weights.shape == (0, 8) and host(r.offsets).tolist() == [0] * 65


def test_one_expert_takes_all():
    x = torch.zeros(5000, 96)
    x[:, 41] = 5.0
    _check(x, 1)
    _check(x, 3, "sigmoid")


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_logits_off_their_vector_alignment(dtype):
    x = _logits(101, 64, 2, dtype)
    flat = torch.empty(101 * 64 + 1, dtype=x.dtype, device="cuda")
    y = flat[1:].view(101, 64)
    y.copy_(x)
    _check(x, 8, r=mx.route(y, 8))
    dw = torch.randn(101, 8)
    e = mx.route(x.cuda(), 8).experts
    assert torch.equal(mx.route_backward(dw.cuda(), y, e), mx.route_backward(dw.cuda(), x.cuda(), e))


def _backward_check(x, e, dw, score, renormalize, scale):
    got = mx.route_backward(dev(dw.astype(np.float32)), x.cuda(), dev(e), score, renormalize, scale)
    assert got.dtype == x.dtype
    x64, dw = x.double().numpy(), dw.astype(np.float32).astype(np.float64)
    ref = P.route_backward(dw, x64, e, score, renormalize, scale)
    # magnitudes of the terms each element is built from
    p = P.scores(x64, score)
    u = np.where(e < 0, 0.0, np.take_along_axis(p, np.maximum(e, 0), 1))
    S = np.maximum(u.sum(1, keepdims=True), 1e-300) if renormalize else 1.0
    a = u / S
    G = (np.abs(dw) * a).sum(1, keepdims=True)
    term = np.abs(scale) * a * (np.abs(dw) + G)
    mag = np.zeros(x64.shape)
    np.add.at(mag, (np.arange(len(e))[:, None], np.maximum(e, 0)), np.where(e < 0, 0.0, term))
    if score == "softmax" and not renormalize:
        mag = mag + np.abs(scale) * p * G
    r = np.abs(x64[np.isfinite(x64)]).max() if np.isfinite(x64).any() else 0.0
    tol = (64 + x64.shape[1] / 16 + 16 * r) * EPS * mag + 1e-37
    if x.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -8)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= tol).all(), (err - tol).max()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (17, 60, 6), (130, 127, 16), (500, 250, 6),
                                   (64, 512, 8), (33, 300, 3), (5000, 64, 8)])
def test_backward(score, renormalize, dtype, T, E, k):
    x = _logits(T, E, T * 3 + E, dtype, mask=0.1 if E > 32 else 0.0)
    e = P.choose(x.double().numpy(), k, score)
    dw = np.random.default_rng(E).normal(size=e.shape)
    _backward_check(x, e, dw, score, renormalize, 1.0)
    _backward_check(x, e, dw, score, renormalize, 2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_backward_matches_differences_of_the_weights(score, renormalize):
    """The GPU's gradient against central differences of the 64-bit weights."""
    x = _logits(3, 12, 1)
    x64 = x.double().numpy()
    e = P.choose(x64, 4, score)
    dw = np.random.default_rng(2).normal(size=e.shape).astype(np.float32)
    got = host(mx.route_backward(dev(dw), x.cuda(), dev(e), score, renormalize, 1.5)).astype(np.float64)
    h = 1e-5
    for t in range(3):
        for i in range(12):
            d = np.zeros_like(x64)
            d[t, i] = h
            diff = (P.weights(x64 + d, e, score, renormalize, 1.5) -
                    P.weights(x64 - d, e, score, renormalize, 1.5))
            # 4 choices, |dw| < 4, weights < 1.5: the 32-bit gradient's terms stay under 24
            assert abs((diff * dw).sum() / (2 * h) - got[t, i]) < 24 * 128 * EPS


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_backward_skips_masked_and_bad_choices(score, renormalize):
    x = _logits(40, 64, 3, mask=0.2)
    x[0] = -float("inf")
    x[1, 2:] = -float("inf")
    e = P.choose(x.double().numpy(), 5, score)
    assert (e[0] == -1).all() and (e[1, 2:] == -1).all()
    dw = np.random.default_rng(6).normal(size=e.shape)
    _backward_check(x, e, dw, score, renormalize, 1.0)
    bad = e.copy()
    bad[2:, 4] = 64                   # outside the experts: as -1
    got = mx.route_backward(dev(dw.astype(np.float32)), x.cuda(), dev(bad), score, renormalize)
    bad[2:, 4] = -1
    want = mx.route_backward(dev(dw.astype(np.float32)), x.cuda(), dev(bad), score, renormalize)
    assert torch.equal(got, want)


def test_runs_on_the_current_stream_and_repeats():
    x = _logits(20000, 128, 4).cuda()
    b = torch.zeros(128, device="cuda")
    want = mx.route(x, 8, "sigmoid", b, n_groups=8, top_groups=4)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            got = mx.route(x, 8, "sigmoid", b, n_groups=8, top_groups=4)
        s.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    say("[route] same bytes on another stream, three times")


def test_refusals():
    x = torch.zeros(4, 8, device="cuda")
    e = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    for call, kind in [
        (lambda: mx.route(x, 0), ValueError), (lambda: mx.route(x, 9), ValueError),
        (lambda: mx.route(x.t(), 2), ValueError), (lambda: mx.route(x[0], 2), ValueError),
        (lambda: mx.route(x, 2, bias=torch.zeros(7, device="cuda")), ValueError),
        (lambda: mx.route(x, 2, bias=x.double()[0]), TypeError),
        (lambda: mx.route(x, 2, n_groups=3), mx.MXError),
        (lambda: mx.route(x, 5, n_groups=4, top_groups=2), mx.MXError),
        (lambda: mx.route(torch.zeros(2, 600, device="cuda"), 2), mx.MXError),
        (lambda: mx.route_backward(w, x, e[:3]), ValueError),
        (lambda: mx.route_backward(w[:, :1].contiguous(), x, e), ValueError),
        (lambda: mx.route_backward(w, x, e.long()), TypeError),
    ]:
        with pytest.raises(kind):
            call()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("value", ["top2", "max"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("E,n", [(64, 4), (60, 4), (256, 2), (512, 2), (200, 8)])
def test_infinite_logits_in_later_groups(score, value, bias, E, n):
    """A group with a +inf logit beats the groups without one, wherever it
    stands: groups of a few chunks, of odd sizes, and of several rows of
    chunks."""
    x = _logits(12, E, E + n, mask=0.2)
    inf, gs = float("inf"), E // n
    x[0, E - 3] = inf                             # in the last group
    x[1, gs + 1] = x[1, E - 1] = inf              # in two groups (in one where there are two)
    x[2, E - 2:] = inf                            # two in one group,
    x[2, 1] = inf                                 # one in another
    x[3] = -inf
    x[3, E - 1] = inf                             # the only expert left
    x[4, E - 1] = inf
    x[4, 0] = float("nan")
    x[5, gs] = inf
    b = torch.from_numpy(np.random.default_rng(2).normal(size=E).astype(np.float32)) if bias else None
    for top_groups in (1, 2):
        for renormalize in (True, False):
            _check(x, 4, score, b, n, top_groups, value, renormalize)


@pytest.mark.parametrize("E,n", [(64, 4), (60, 4), (256, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_that_underflow_add_nothing_to_a_group(score, E, n):
    """Scores below 2^-1075 are 0 in 64 bits: a group of two such is worth no
    more than a group of one, and the lower index wins."""
    gs = E // n
    x = torch.full((4, E), -float("inf"))
    x[:, -1] = 0.0                                # the last group's score is not 0
    x[0, 0] = x[1, 1] = -800.0                    # group 0: one score of 0
    if n > 2:
        x[0, gs] = x[0, gs + 1] = -850.0          # group 1: two
        x[1, gs:2 * gs] = torch.finfo(torch.float32).min
    x[2, :gs] = -2000.0
    x[3, 0] = -700.0                              # e^-700 > 2 e^-701, both above 2^-1022
    if n > 2:
        x[3, gs] = x[3, gs + 1] = -701.0
    for bias in (None, torch.zeros(E)):
        _check(x, 3, score, bias, n, 2)
    if score == "softmax" and n > 2:              # e^-720 > 2 e^-725, both below 2^-1022
        x = torch.full((2, E), -float("inf"))
        x[:, -1] = 0.0
        x[0, 0] = x[1, gs] = -720.0
        x[0, gs] = x[0, gs + 1] = x[1, 0] = x[1, 1] = -725.0
        _check(x, 3, score, None, n, 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,n,tn", [
    (700, 64, 8, 1, 1), (1500, 256, 8, 8, 4), (333, 60, 5, 6, 2), (200, 512, 12, 1, 1),
])
def test_bfloat16_logits_with_a_bias(score, T, E, k, n, tn):
    """BF16 logits tie often; the bias orders what they leave equal."""
    x = _logits(T, E, T + E, "bfloat16", mask=0.05)
    bias = torch.from_numpy((0.05 * np.random.default_rng(k).normal(size=E)).astype(np.float32))
    _check(x, k, score, bias, n, tn, scale=2.5)
    _check(x, k, score, bias, n, tn, "max", renormalize=False)
    _check(x, k, score, (bias * 64).round() / 64, n, tn)    # a bias of few values: ties again


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_groups_with_a_bias_over_many_workgroups(dtype):
    x = _logits(20011, 128, 6, dtype, mask=0.02)
    bias = torch.from_numpy((0.1 * np.random.default_rng(3).normal(size=128)).astype(np.float32))
    _check(x, 8, "sigmoid", bias, 8, 4, scale=2.5)
    _check(x, 6, "softmax", bias, 4, 2)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,n", [(128, 2), (256, 2), (512, 2), (512, 4), (192, 3)])
def test_groups_of_several_rows_of_chunks(score, E, n):
    """Groups longer than the lanes of a token hold side by side."""
    x = _logits(300, E, n, mask=0.1)
    bias = torch.from_numpy((0.1 * np.random.default_rng(E).normal(size=E)).astype(np.float32))
    for b in (None, bias):
        for value in ("top2", "max"):
            _check(x, 8, score, b, n, n - 1, value)
            _check(x, 12, score, b, n, 1, value)
