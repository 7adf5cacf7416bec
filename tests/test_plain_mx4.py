"""Pins of the plain 64-bit reference of 4-bit weights and 8-bit checkpoints:
closed forms, brute force, torch's casts and differences (CPU)."""
import numpy as np
import torch

import oracle
import plain_mx4 as P


def test_e2m1_codes():
    assert P.grid_values("e2m1").tolist() == [0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6]


def test_fp8_codes_are_torchs():
    for elem, kind in (("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)):
        want = torch.arange(256, dtype=torch.uint8).view(kind).double().numpy()
        np.testing.assert_array_equal(P.grid_values(elem), want)


def test_encode_against_a_search():
    g = P.grid_values("e2m1")[:8]
    v = np.concatenate([np.linspace(0, 6, 1537), [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 1e-9, 5.999]])
    for x, c in zip(v, P.encode(v, "e2m1")):
        d = np.abs(g - x)
        best = np.flatnonzero(d == d.min())
        assert c == (best[0] if len(best) == 1 else best[best % 2 == 0][0]), (x, c)
    assert P.encode(np.array([-0.25, -5.0, -6.0, 7.0]), "e2m1").tolist() == [8, 14, 15, 7]


def test_scale_exponents():
    for elem, (big, _, _) in P.FORMAT.items():
        for k in (-100, -1, 0, 3, 90):
            assert P.scale_exponent(big * 2.0 ** k, elem) == k
            assert P.scale_exponent(np.nextafter(big * 2.0 ** k, np.inf), elem) == k + 1
        assert P.scale_exponent(0.0, elem) == -127
        assert P.scale_exponent(2.0 ** -133, elem) == -127


def test_eight_bit_rows_are_the_oracles():
    g = torch.Generator().manual_seed(1)
    x = (torch.randn((40, 96), generator=g) * torch.exp(3 * torch.randn((40, 1), generator=g))).to(torch.bfloat16)
    x[3] = 0
    x[5, 7] = float("inf")
    x[6, 40] = float("nan")
    bits = x.view(torch.int16).numpy().view(np.uint16)
    for elem in ("e4m3", "e5m2"):
        q, s = P.quant_rows(P.bf16_values(bits), elem)
        oq, os_ = oracle.quant_row(bits, elem=elem)
        np.testing.assert_array_equal(q, oq)
        np.testing.assert_array_equal(s, os_)


def test_pack_order():
    codes = np.arange(32, dtype=np.uint8)[None] % 16
    assert P.pack(codes)[0, :3].tolist() == [0x10, 0x32, 0x54]
    np.testing.assert_array_equal(P.unpack(P.pack(codes)), codes)


def test_values_of_a_block():
    q = np.zeros((1, 16), np.uint8)
    q[0, 0], q[0, 15] = 0xF1, 0x70            # 0.5, -6 ... 0, 6
    v = P.values(q, np.array([[129]], np.uint8), "e2m1")[0]
    assert v[0] == 2.0 and v[1] == -24.0 and v[30] == 0 and v[31] == 24.0
    assert np.isnan(P.values(q, np.array([[255]], np.uint8), "e2m1")).all()


def test_bf16_round():
    x = np.random.default_rng(0).standard_normal(4000) * 10.0 ** np.random.default_rng(1).integers(-39, 38, 4000)
    x = x.astype(np.float32).astype(np.float64)
    np.testing.assert_array_equal(P.bf16_round(x), torch.from_numpy(x).float().to(torch.bfloat16).double().numpy())
    assert P.bf16_round(3.4e38) == np.inf and P.bf16_round(1 + 2.0 ** -8) == 1.0


def test_swiglu_against_torch_and_its_gradient():
    rng = np.random.default_rng(2)
    x, dh = rng.standard_normal((7, 64)) * 3, rng.standard_normal((7, 32))
    t = torch.from_numpy(x).requires_grad_()
    h = torch.nn.functional.silu(t[:, :32]) * t[:, 32:]
    np.testing.assert_allclose(P.swiglu(x), h.detach().numpy(), rtol=1e-13, atol=1e-15)
    h.backward(torch.from_numpy(dh))
    np.testing.assert_allclose(P.swiglu_backward(dh, x), t.grad.numpy(), rtol=1e-12, atol=1e-14)


def test_swiglu_gradient_against_differences():
    rng = np.random.default_rng(3)
    x, dh, eps = rng.standard_normal((3, 64)) * 2, rng.standard_normal((3, 32)), 1e-6
    got = P.swiglu_backward(dh, x)
    for i in range(3):
        for j in range(0, 64, 5):
            up, dn = x.copy(), x.copy()
            up[i, j] += eps
            dn[i, j] -= eps
            want = ((P.swiglu(up) - P.swiglu(dn)) * dh).sum() / (2 * eps)
            # the difference's own error: eps^2 of the third derivative, and
            # 2^-52 of sums below 100 over eps
            assert abs(got[i, j] - want) < 1e-7
