"""Pins of the 64-bit dense-expert oracle: E4M3 rounding against the format's own list of values,
block scales, the block product against an explicit triple sum, SwiGLU's gradients against
differences."""
import numpy as np
import torch

from oracle import dense as OD


def e4m3_values():
    """Every finite E4M3 value from its definition: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    v = []
    for e in range(16):
        for m in range(8):
            if e == 15 and m == 7:
                continue                                   # NaN
            v.append((m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7))
    return np.array(sorted(v))


def test_rounding_is_the_nearest_value_with_ties_to_the_even_mantissa():
    vals = e4m3_values()
    assert vals[-1] == 448.0 and vals[1] == 2.0 ** -9
    np.testing.assert_array_equal(OD.e4m3_round(vals), vals)
    mids = (vals[1:] + vals[:-1]) / 2
    for i, mid in enumerate(mids):
        # consecutive values alternate even and odd mantissas, value 0 being even
        assert OD.e4m3_round(mid) == vals[i if i % 2 == 0 else i + 1]
        assert OD.e4m3_round(-mid) == -vals[i if i % 2 == 0 else i + 1]
        assert OD.e4m3_round(mid * (1 + 1e-9)) == vals[i + 1]
        assert OD.e4m3_round(mid * (1 - 1e-9)) == vals[i]
    assert np.isnan(OD.e4m3_round(np.inf)) and np.isnan(OD.e4m3_round(np.nan))
    rng = np.random.default_rng(1)
    x = rng.standard_normal(20000) * np.exp2(rng.integers(-12, 8, 20000))
    x = x[np.abs(x) <= 448].astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).to(torch.float64).numpy()
    np.testing.assert_array_equal(OD.e4m3_round(x), want)


def test_block_scales_put_the_largest_value_at_most_448():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 300)) * np.exp2(rng.integers(-20, 20, (5, 1)))
    x[3, :128] = 0.0
    x[4, 130] = np.inf
    s = OD.block_scales(x)
    assert s.shape == (5, 3) and s[3, 0] == 1.0
    for i in range(5):
        for j in range(3):
            b = np.abs(x[i, 128 * j:128 * (j + 1)])
            top = b[np.isfinite(b)].max()
            if top:
                assert top / s[i, j] <= 448.0 < 2 * top / s[i, j]
    s = OD.block_scales(rng.standard_normal((200, 130)), 128)
    assert s.shape == (2, 2)


def test_block_product_is_the_explicit_sum():
    rng = np.random.default_rng(3)
    M, N, K = 3, 130, 160
    q_x, s_x = OD.quantize(rng.standard_normal((M, K)))
    q_w, s_w = OD.quantize(rng.standard_normal((N, K)), 128)
    got, mag = OD.block_product(q_x, s_x, q_w, s_w)
    for m in range(M):
        for n in range(0, N, 43):
            want = sum(s_x[m, k // 128] * s_w[n // 128, k // 128] * q_x[m, k] * q_w[n, k] for k in range(K))
            assert abs(want - got[m, n]) <= 1e-12 * mag[m, n]


def test_swiglu_gradients_against_differences():
    rng = np.random.default_rng(4)
    T, D, F = 4, 6, 5
    x, a, b, dh = (rng.standard_normal(s) for s in ((T, D), (F, D), (F, D), (T, F)))

    def loss(x, a, b):
        return float((OD.swiglu(x, a, b)[0] * dh).sum())

    _, g, u = OD.swiglu(x, a, b)
    dg, du = OD.swiglu_factor_grads(g, u, dh)
    grads = OD.swiglu_grads(dg, du, x, a, b)
    step = 1e-5
    for which, grad in enumerate(grads):
        arrays = [x, a, b]
        for idx in np.ndindex(*arrays[which].shape):
            up, down = [v.copy() for v in arrays], [v.copy() for v in arrays]
            up[which][idx] += step
            down[which][idx] -= step
            diff = (loss(*up) - loss(*down)) / (2 * step)
            # central difference: step^2 / 6 third derivatives (below 10 here), and 1e-16 / step rounding
            assert abs(diff - grad[idx]) <= 1e-8 * (1 + abs(diff))
