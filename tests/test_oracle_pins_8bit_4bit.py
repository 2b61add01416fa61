"""Pins of the oracle's e4m3 moments and MX4 weight: hand values, brute force, invariants."""
import numpy as np
import pytest
import torch

import oracle as O


# ------------------------------------------------------------------------------- e4m3 moments
def test_e4m3_values_match_torch():
    v = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(O.e4m3_values(), v.astype(np.float64))


def test_moments_to_nearest_are_the_nearest_code():
    rng = np.random.default_rng(0)
    x = rng.normal(size=700) * np.exp2(rng.integers(-30, 0, 700))
    q, u = O.e4m3_moments(x, False)
    vals = O.e4m3_values()
    vals = np.sort(vals[np.isfinite(vals)])
    for i in range(700):
        y = x[i] / u[i // 256]
        assert abs(q[i] - y) <= np.min(np.abs(vals - y)) * (1 + 1e-12) + 1e-15
    assert u.size == 3 and np.allclose(u[0], np.abs(x[:256]).max() / 448)
    assert np.abs(q[:256]).max() == 448


def test_roots_of_second_moments_never_round_to_zero():
    x = np.array([1.0, 1e-9, 0.0, 2.0 ** -12])
    q, u = O.e4m3_moments(x, True)
    assert q[1] == 2.0 ** -9 and q[2] == 0 and q[0] == 448
    assert O.e4m3_moments(x, False)[0][1] == 0
    # not finite: NaN of its own, not of its block; a block below 2^-100 is zeros
    q, u = O.e4m3_moments(np.array([1.0, np.inf, np.nan]), False)
    assert q[0] == 448 and np.isnan(q[1]) and np.isnan(q[2]) and u[0] == 1 / 448
    assert not O.e4m3_moments(np.full(5, 1e-31), False)[0].any()


def test_stochastic_rounding_is_unbiased_and_stays_next_to_the_value():
    # 65536 equidistant draws: the mean of floor(k + r/65536) is k within 2^-16 of a step.
    r = np.arange(65536.0)
    for a in (300.0, 17.3, 0.02, 0.003, 0.0001):
        g = float(O.e4m3_grid(np.array(a)))
        x = np.zeros(65536 // 255 * 256 + 512)
        q = np.floor(a / g + r / 65536) * g
        assert abs(q.mean() - a) <= g * 2.0 ** -16
        assert set(np.unique(q)) <= {np.floor(a / g) * g, np.floor(a / g) * g + g}
    h = O.element_bits(1 << 16, 3, 12345)
    assert h.max() < 2 ** 32
    # Uniform halves, independent of each other, of the tensor and of the seed: standard
    # deviations of a mean of 65536 uniforms (1/sqrt(12)/256 = 1.1e-3), six of them allowed.
    lo, hi = (h & np.uint64(0xFFFF)) / 65536.0, (h >> np.uint64(16)) / 65536.0
    assert abs(lo.mean() - 0.5) < 7e-3 and abs(hi.mean() - 0.5) < 7e-3
    for other in (hi, np.roll(lo, 1), (O.element_bits(1 << 16, 4, 12345) & np.uint64(0xFFFF)) / 65536.0,
                  (O.element_bits(1 << 16, 3, 12346) & np.uint64(0xFFFF)) / 65536.0,
                  (O.element_bits(1 << 16, 3, 12345 + (1 << 32)) & np.uint64(0xFFFF)) / 65536.0):
        assert abs(np.corrcoef(lo, other)[0, 1]) < 6 / 256
    assert np.corrcoef(lo, lo)[0, 1] == pytest.approx(1)


def test_bf16_stochastic_stays_on_the_grid():
    h = O.element_bits(4096, 0, 9)
    p = np.random.default_rng(1).normal(size=4096)
    q = O.bf16_stochastic(p, h)
    assert np.array_equal(torch.tensor(q).to(torch.bfloat16).double().numpy(), q)
    assert np.all(np.abs(q - p) < np.abs(p) * 2.0 ** -7) and abs(np.mean((q - p) / np.abs(p))) < 3e-4


# ---------------------------------------------------------------------------------- MX4 weight
def test_mx4_hand_example():
    # absmax 6 -> scale 2^0: every code's value, every tie (to the even code), saturation.
    w = np.zeros((3, 32))
    w[0, :16] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, 0.24, 0.26, -6, 7.9, -0.0, 5.01]
    w[1, 0], w[1, 1] = 2.0 ** -127, np.nan
    w[2, 0], w[2, 1] = 96.0, 1.0
    c, s = O.mx4_quantize(w)
    nib = np.stack([c & 15, c >> 4], 2).reshape(3, 32)
    # 7.9 has exponent 2, so the scale is still 2^0 and 7.9 saturates at 6.
    assert s[0, 0] == 127 and list(nib[0, :16]) == [7, 0, 2, 2, 4, 4, 6, 6, 8, 10, 0, 1, 15, 7, 8, 7]
    assert s[1, 0] == 255 and not nib[1].any() and np.isnan(O.mx4_dequantize(c, s)[1]).all()
    assert s[2, 0] == 127 + 4 and O.mx4_dequantize(c, s)[2, 0] == 96 and nib[2, 1] == 0  # 1/16 scale: below 1/4
    zero = O.mx4_quantize(np.zeros((1, 64)))
    assert not zero[0].any() and not zero[1].any()


def test_mx4_nearest_by_brute_force_and_invariants():
    rng = np.random.default_rng(5)
    W = rng.normal(size=(9, 96)) * np.exp2(rng.integers(-8, 8, (9, 1)))
    c, s = O.mx4_quantize(W)
    V = O.mx4_dequantize(c, s)
    grid = np.concatenate([O.mx4_dequantize(np.arange(256, dtype=np.uint8).reshape(16, 16), np.full((16, 1), 127, np.uint8)).ravel()])
    grid = np.unique(grid)
    sc = np.repeat(np.exp2(s.astype(float) - 127), 32, axis=1)
    for i in range(9):
        for j in range(96):
            y = np.clip(W[i, j] / sc[i, j], -6, 6)
            assert abs(V[i, j] / sc[i, j] - y) == np.min(np.abs(grid - y))
    # on-grid rows come back exactly; odd symmetry; power-of-two invariance
    c2, s2 = O.mx4_quantize(V)
    assert np.array_equal(O.mx4_dequantize(c2, s2), V)
    assert np.array_equal(O.mx4_dequantize(*O.mx4_quantize(-W)), -V)
    assert np.array_equal(O.mx4_dequantize(*O.mx4_quantize(W * 1024)), V * 1024)


def test_mx4_merge_with_zero_theta_is_a_fixed_point():
    rng = np.random.default_rng(2)
    b, P = 32, 32 * 31 // 2
    c, s = O.mx4_quantize(rng.normal(size=(64, 96)) * 0.02)
    pL, pR = rng.permutation(64), rng.permutation(96)
    Wn, cn, sn, tR, tP = O.mx4_merge(c, s, np.zeros((2, P)), np.zeros((3, P)), pL, pR, pL, pR, b, 3)
    assert np.array_equal(Wn, O.mx4_dequantize(c, s)) and np.array_equal(O.mx4_dequantize(cn, sn), Wn)
    assert not tR.any() and not tP.any()


@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("a", [448.0, 447.9, 300.0, 17.3, 1.0, 0.02, 2.0 ** -6, 0.0117, 0.003, 0.0021, 0.0001])
def test_moments_rounded_stochastically_are_unbiased(positive, a):
    # Blocks whose first element, 448, makes the scale 1, so that the other 255 stand on the grid as they are; 65536 equidistant
    # draws over them.  floor(a / g + r / 65536) is up for a fraction of the draws that is a / g's own within one draw,
    # so the mean is a within 2^-16 of a step (2^-40 of a more for the scale's own division).
    n = 65536
    r = np.zeros((258, 256))
    r[:, 1:] = np.resize(np.arange(n, dtype=float), (258, 255))
    for sign in ((1.0,) if positive else (1.0, -1.0)):
        x = np.full((258, 256), sign * a)
        x[:, 0] = 448.0
        q, u = O.e4m3_moments(x.ravel(), positive, r.ravel())
        assert np.array_equal(u, np.ones(258))
        q = q.reshape(258, 256)
        assert np.all(q[:, 0] == 448)
        q = q[:, 1:].ravel()[:n] * sign
        vals = O.e4m3_values()
        vals = np.unique(np.abs(vals[np.isfinite(vals)]))
        lo, hi = vals[vals <= a][-1], vals[vals >= a][0]
        if positive and lo == 0:  # never stored as zero
            assert np.all(q == hi) and hi == 2.0 ** -9
            continue
        assert set(np.unique(q)) <= {lo, hi}
        assert abs(q.mean() - a) <= (hi - lo) * 2.0 ** -16 + a * 2.0 ** -40
        assert a in (lo, hi) or {lo, hi} == set(np.unique(q))  # exact values stay, others go both ways


def test_moments_of_zero_stay_zero_under_any_draw():
    x = np.zeros(256)
    x[0] = 1.0
    for positive in (False, True):
        q, _ = O.e4m3_moments(x, positive, np.full(256, 65535.0))
        assert q[0] == 448 and not q[1:].any()


def test_element_bits_go_on_past_32_bits():
    # One formula for every position: a later start continues the sequence, and past 2^32 it does not repeat.
    a = O.element_bits(1000, 2, 77)
    assert np.array_equal(O.element_bits(600, 2, 77, start=400), a[400:])
    far = O.element_bits(1000, 2, 77, start=(1 << 32) - 500)
    assert not np.array_equal(far[500:], a[:500])
    # By hand: element 2^32 + 1 of tensor 0 under seed 0 (salt 0xBB67AE85).
    M = 0xFFFFFFFF
    h = (0x9E3779B1 + 0xBB67AE85 + 0x6A09E667) & M
    h = ((h ^ (h >> 16)) * 0x6A09E667) & M
    h = ((h ^ (h >> 15)) * 0xBB67AE85) & M
    assert int(O.element_bits(1, 0, 0, start=(1 << 32) + 1)[0]) == h ^ (h >> 16)
