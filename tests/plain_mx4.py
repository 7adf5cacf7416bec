"""Plain 64-bit reference of the 4-bit weights and 8-bit checkpoints: codes and
scales from the formats' definitions, products, SwiGLU and its gradient.
numpy only; no code shared with the library."""
import numpy as np

# largest finite value, mantissa bits, exponent of the smallest normal value
FORMAT = {"e4m3": (448.0, 3, -6), "e5m2": (57344.0, 2, -14), "e2m1": (6.0, 1, 0)}
NAN_PAYLOAD = {"e4m3": 0x7F, "e5m2": 0x7F, "e2m1": 7}


def grid_values(elem):
    """Value of every code (index = code), sign bit included; NaN and infinity
    where the format has them."""
    big, bits, low = FORMAT[elem]
    n = 8 if elem == "e2m1" else 128
    v = np.empty(n)
    for c in range(n):
        m, e = c & ((1 << bits) - 1), c >> bits
        v[c] = m * 2.0 ** (low - bits) if e == 0 else (1 + m / (1 << bits)) * 2.0 ** (low + e - 1)
    if elem == "e4m3":
        v[127] = np.nan
    if elem == "e5m2":
        v[124], v[125:] = np.inf, np.nan
    return np.concatenate([v, -v])


def bf16_values(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def bf16_round(x):
    """Nearest BF16 value of a float64, ties to even, as float64."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        e = np.clip(np.frexp(np.where(np.isfinite(x), x, 1.0))[1] - 1, -126, None)
        step = np.ldexp(1.0, e - 7)
        r = np.rint(x / step) * step
        r = np.where(np.abs(r) >= 2.0 ** 128, np.copysign(np.inf, x), r)
    return np.where(np.isfinite(x), r, x)


def to_bf16_bits(x):
    """Bits of values that BF16 holds exactly."""
    return (np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def scale_exponent(amax, elem):
    """Smallest e with amax <= big 2^e, clamped; zero gives -127."""
    big = FORMAT[elem][0]
    m, e = np.frexp(np.asarray(amax, np.float64) / big)
    e = np.where(m == 0.5, e - 1, e)
    return np.clip(np.where(np.asarray(amax) == 0, -127, e), -127, 127).astype(np.int64)


def encode(v, elem):
    """Codes of v (already over the scale), nearest with ties to even, saturating."""
    g = grid_values(elem)
    half = g[:len(g) // 2]
    half = half[np.isfinite(half)]
    a = np.minimum(np.abs(v), half[-1])
    hi = np.clip(np.searchsorted(half, a), 1, len(half) - 1)
    lo = hi - 1
    dl, dh = a - half[lo], half[hi] - a
    code = np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
    return (code + np.where(np.signbit(v), len(g) // 2, 0)).astype(np.uint8)


def pack(codes):
    return codes[..., ::2] | (codes[..., 1::2] << 4)


def unpack(q):
    return np.stack([q & 15, q >> 4], -1).reshape(q.shape[:-1] + (2 * q.shape[-1],))


def quant_rows(x, elem):
    """x float64 [..., C] -> (payload, scale bytes), blocks along the last axis."""
    b = x.reshape(x.shape[:-1] + (-1, 32))
    bad = ~np.isfinite(b).all(-1)
    amax = np.abs(np.where(np.isfinite(b), b, 0.0)).max(-1)
    e = scale_exponent(amax, elem)
    codes = encode(np.where(bad[..., None], 0.0, b) * np.ldexp(1.0, -e)[..., None], elem)
    codes = np.where(bad[..., None], NAN_PAYLOAD[elem], codes).astype(np.uint8).reshape(x.shape)
    s = np.where(bad, 255, e + 127).astype(np.uint8)
    return (pack(codes) if elem == "e2m1" else codes), s


def values(q, s, elem):
    """float64 values of an MX tensor in row blocks."""
    codes = unpack(q) if elem == "e2m1" else q
    v = grid_values(elem)[codes].reshape(s.shape + (32,))
    with np.errstate(invalid="ignore"):
        v = v * np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(np.int64) - 127))[..., None]
    return v.reshape(codes.shape)


def gemm(a, sa, b, sb, a_elem):
    """(result, sum of |products|) of C = A B^T."""
    x, y = values(a, sa, a_elem), values(b, sb, "e2m1")
    return x @ y.T, np.abs(x) @ np.abs(y).T


def gemm_tolerance(ref, absum, K, a_elem):
    """An FP32 sum is off by at most a step (2^-23) of the sum of magnitudes
    for each of its K terms, and the result's rounding by half a BF16 step.

    With an 8-bit operand the matrix instruction adds eight neighbouring
    products at a time, on the exponent of the largest: bits at 2^-14 of that
    power of two and below are dropped (448 - 448 + 15/64 in one group of eight
    gives 14/64, and 15/64 exactly where the small one stands in the next group;
    57344 - 57344 + 14 gives 12).  The largest keeps all its bits; each of the
    other seven loses less than 2^-13 of it, and it is at most the group's sum of
    magnitudes: 7 2^-13 of that sum for the group, hence of absum for all of
    them.  Products of two 4-bit codes span 7 bits and lose none."""
    acc = (K * 2.0 ** -23 + (0.0 if a_elem == "e2m1" else 7 * 2.0 ** -13)) * absum
    return 2.0 ** -8 * (np.abs(ref) + acc) + acc + 2.0 ** -134


def sigmoid(g):
    t = np.exp(-np.abs(g))
    return np.where(g >= 0, 1 / (1 + t), t / (1 + t))


def swiglu(x):
    F = x.shape[1] // 2
    g, u = x[:, :F], x[:, F:]
    return g * sigmoid(g) * u


def swiglu_backward(dh, x):
    F = dh.shape[1]
    g, u = x[:, :F], x[:, F:]
    p = sigmoid(g)
    return np.concatenate([dh * u * p * (1 + g * (1 - p)), dh * g * p], 1)


# FP32 evaluation of sigmoid for |g| <= 16: the exponent's argument is off by
# half a step of a product up to 16 log2(e) < 32 (2^-20 of the exponential),
# the exponential, reciprocal and the product of two by 2^-23 each; g, u and dh
# multiply on with half a step each.  Together under 2^-18.
ACT_EPS = 2.0 ** -18


def swiglu_backward_tolerance(dh, x):
    """Half a BF16 step of the result, and the FP32 evaluation, whose error is
    relative to the terms of 1 + g (1 - p)."""
    F = dh.shape[1]
    g, u = x[:, :F], x[:, F:]
    p = sigmoid(g)
    mag = np.concatenate([np.abs(dh * u) * p * (1 + np.abs(g) * (1 - p)), np.abs(dh * g) * p], 1)
    return 2.0 ** -8 * np.abs(swiglu_backward(dh, x)) + ACT_EPS * mag + 2.0 ** -133


def bf16_decided(x):
    """Whether every value within ACT_EPS of x rounds to the same BF16."""
    return bf16_round(x * (1 - ACT_EPS)) == bf16_round(x * (1 + ACT_EPS))
