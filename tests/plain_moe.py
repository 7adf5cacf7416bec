"""Plain 64-bit implementations of routing, token movement and gradient
clipping (numpy, from the definitions; nothing shared with the HIP library)."""
import numpy as np

NEG = -np.inf


def scores(x, score):
    """Router scores of logits x [T, E] in 64 bits.  A NaN takes no part in a
    row's sum; of several +inf logits each gets an equal share."""
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        m = np.nanmax(np.where(np.isnan(x), NEG, x), axis=1, keepdims=True)
        z = np.where(x == m, 1.0, np.exp(x - m))
        z = np.where(np.isneginf(x), 0.0, z)
        tot = np.nansum(z, axis=1, keepdims=True)
        return z / np.where(tot > 0, tot, 1.0)


def _order(v):
    """Columns of v by falling value: numbers, then NaN, then -inf (masked),
    equal ones by index."""
    cls = np.where(np.isneginf(v), 2, np.where(np.isnan(v), 1, 0))
    key = np.where(cls == 0, -v, 0.0)
    first = np.argsort(key, axis=1, kind="stable")
    cls2 = np.take_along_axis(cls, first, 1)
    second = np.argsort(cls2, axis=1, kind="stable")
    return np.take_along_axis(first, second, 1)


def choose(x, k, score, bias=None, n_groups=1, top_groups=1, group_value="top2"):
    """experts [T, k], -1 where none is left."""
    T, E = x.shape
    # without a bias experts are in their logits' order, which the scores keep
    v = np.where(np.isneginf(x), NEG, x)
    value = scores(x, score)
    if bias is not None:
        with np.errstate(all="ignore"):
            v = value = np.where(np.isneginf(x), NEG, value + bias)
    if n_groups > 1:
        by = v.reshape(T * n_groups, E // n_groups)
        o = _order(by)
        best = np.take_along_axis(by, o[:, :1], 1)[:, 0]
        val = best
        if group_value == "top2":
            vals = np.where(np.isneginf(v), NEG, value).reshape(by.shape)
            val = np.take_along_axis(vals, o[:, :1], 1)[:, 0]
            if E // n_groups > 1:
                second = np.take_along_axis(vals, o[:, 1:2], 1)[:, 0]
                with np.errstate(all="ignore"):
                    val = np.where(np.isneginf(second), val, val + second)
        rank = np.argsort(_order(val.reshape(T, n_groups)), axis=1)
        v = np.where(np.repeat(rank < top_groups, E // n_groups, axis=1), v, NEG)
    o = _order(v)[:, :k]
    return np.where(np.isneginf(np.take_along_axis(v, o, 1)), -1, o).astype(np.int32)


def weights(x, experts, score, renormalize, scale):
    """Weights of the chosen experts; renormalised ones in a form that holds
    where every chosen score underflows."""
    none = experts < 0
    xe = np.take_along_axis(x, np.maximum(experts, 0), 1)
    with np.errstate(all="ignore"):
        if renormalize:
            top = np.where(none | np.isnan(xe), NEG, xe).max(1, keepdims=True)
            if score == "softmax":
                u = np.where(xe == top, 1.0, np.exp(xe - top))
            else:
                s = np.minimum(top, 0.0)
                u = 1.0 / (np.exp(s) + np.exp(s - xe))
            u = np.where(none, 0.0, u)
            w = u / u.sum(1, keepdims=True)
        else:
            w = np.take_along_axis(scores(x, score), np.maximum(experts, 0), 1)
    if score == "softmax":
        w = np.where(np.isnan(x).any(1)[:, None], np.nan, w)
    return np.where(none, 0.0, scale * w)


def layout(experts, E):
    """offsets [E + 1], slots [T, k] of a stable sort of the choices."""
    flat = experts.ravel()
    slots = np.full(flat.size, -1, np.int32)
    kept = np.flatnonzero(flat >= 0)
    kept = kept[np.argsort(flat[kept], kind="stable")]
    slots[kept] = np.arange(kept.size, dtype=np.int32)
    counts = np.bincount(flat[flat >= 0], minlength=E)
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int64), slots.reshape(experts.shape)


def route_backward(dw, x, experts, score, renormalize, scale):
    """dlogits [T, E] = (d weights / d logits)^T dw, through the Jacobians of
    the scores and the renormalisation.  Renormalised softmax weights are the
    softmax of the chosen logits alone, so the other experts' gradient is 0."""
    T, E = x.shape
    none = experts < 0
    idx = np.maximum(experts, 0)
    if score == "softmax" and renormalize:
        a = scores(np.where(none, NEG, np.take_along_axis(x, idx, 1)), score)
        g = np.where(none, 0.0, scale * dw)
        dx = np.zeros((T, E))
        np.add.at(dx, (np.arange(T)[:, None], idx), a * (g - (a * g).sum(1, keepdims=True)))
        return dx
    p = scores(x, score)
    u = np.where(none, 0.0, np.take_along_axis(p, idx, 1))
    g = np.where(none, 0.0, scale * dw)
    if renormalize:
        S = u.sum(1, keepdims=True)
        S = np.where(S > 0, S, 1.0)
        g = np.where(none, 0.0, g / S - (g * u).sum(1, keepdims=True) / (S * S))
    dp = np.zeros((T, E))
    np.add.at(dp, (np.arange(T)[:, None], idx), g)
    if score == "sigmoid":
        return dp * p * (1.0 - p)
    return p * (dp - (dp * p).sum(1, keepdims=True))


def dispatch(x, slots):
    T, k = slots.shape
    y = np.zeros((T * k, x.shape[1]), x.dtype)
    for j in range(k):
        on = slots[:, j] >= 0
        y[slots[on, j]] = x[on]
    return y


def combine(y, slots, w=None, residual=None):
    """(out, sum of magnitudes) in 64 bits."""
    T, k = slots.shape
    out = np.zeros((T, y.shape[1])) if residual is None else residual.astype(np.float64).copy()
    mag = np.abs(out)
    for j in range(k):
        on = slots[:, j] >= 0
        part = y[slots[on, j]].astype(np.float64) * (1.0 if w is None else w[on, j:j + 1])
        out[on] += part
        mag[on] += np.abs(part)
    return out, mag


def combine_backward(dout, y, slots, w):
    """(dy, dweights, sum of magnitudes of each dweight) in 64 bits."""
    T, k = slots.shape
    dy = np.zeros(y.shape)
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for j in range(k):
        on = slots[:, j] >= 0
        dy[slots[on, j]] = w[on, j:j + 1] * dout[on]
        prod = dout[on] * y[slots[on, j]]
        dw[on, j], mag[on, j] = prod.sum(1), np.abs(prod).sum(1)
    return dy, dw, mag


def grad_clip(tensors, max_norm):
    """(norm, clipped tensors) in 64 bits."""
    norm = np.sqrt(sum(float((t * t).sum()) for t in tensors))
    with np.errstate(all="ignore"):
        coef = np.float64(max_norm) / (norm + 1e-6)
        coef = 1.0 if coef >= 1.0 else coef
        return norm, [t * coef for t in tensors]
