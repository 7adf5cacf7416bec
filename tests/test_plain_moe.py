"""The plain 64-bit implementations the GPU tests compare with, pinned on the
CPU: hand-worked choices, and gradients against central differences."""
import numpy as np
import pytest

import plain_moe as P


def test_choice_by_hand():
    x = np.array([[1.0, 3.0, 3.0, -np.inf, 2.0, np.nan]])
    assert P.choose(x, 4, "softmax").tolist() == [[1, 2, 4, 0]]
    assert P.choose(x, 6, "sigmoid").tolist() == [[1, 2, 4, 0, 5, -1]]
    # groups {0,1}, {2,3}, {4,5}: best two sum to 4, 3 (one unmasked), NaN
    assert P.choose(x, 2, "softmax", n_groups=3, top_groups=1, group_value="max").tolist() == [[1, 0]]
    # the bias decides, the weights do not see it
    x = np.array([[0.0, 0.1, 0.2]])
    e = P.choose(x, 1, "sigmoid", bias=np.array([1.0, 0.0, 0.0]))
    assert e.tolist() == [[0]]
    assert P.weights(x, e, "sigmoid", False, 2.0)[0, 0] == pytest.approx(1.0)


def test_layout_by_hand():
    e = np.array([[2, 0], [0, -1], [2, 1]], np.int32)
    off, slots = P.layout(e, 4)
    assert off.tolist() == [0, 2, 3, 5, 5]
    assert slots.tolist() == [[3, 0], [1, -1], [4, 2]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_gradient_matches_differences(score, renormalize):
    rng = np.random.default_rng(3)
    x = rng.normal(size=(4, 7))
    e = P.choose(x, 3, score)
    e[1, 2] = -1
    dw = rng.normal(size=e.shape)
    got = P.route_backward(dw, x, e, score, renormalize, 1.7)
    h = 1e-5
    for t in range(4):
        for i in range(7):
            up, dn = x.copy(), x.copy()
            up[t, i] += h
            dn[t, i] -= h
            d = (P.weights(up, e, score, renormalize, 1.7) - P.weights(dn, e, score, renormalize, 1.7))
            # central differences: h^2 of the third derivative, 2^-53 / h of rounding
            assert abs((d * dw).sum() / (2 * h) - got[t, i]) < 1e-8


def test_combine_gradient_matches_differences():
    rng = np.random.default_rng(4)
    e = np.array([[1, 0], [0, -1], [2, 1]], np.int32)
    _, slots = P.layout(e, 3)
    y, w, dout = rng.normal(size=(6, 5)), rng.random(size=(3, 2)), rng.normal(size=(3, 5))
    dy, dw, _ = P.combine_backward(dout, y, slots, w)
    f = lambda yy, ww: (P.combine(yy, slots, ww)[0] * dout).sum()  # noqa: E731
    h = 1e-4
    for i in np.ndindex(*y.shape):
        d = np.zeros_like(y)
        d[i] = h
        assert abs((f(y + d, w) - f(y - d, w)) / (2 * h) - dy[i]) < 1e-9
    for i in np.ndindex(*w.shape):
        d = np.zeros_like(w)
        d[i] = h
        assert abs((f(y, w + d) - f(y, w - d)) / (2 * h) - dw[i]) < 1e-9
