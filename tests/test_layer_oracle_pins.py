"""The oracle of the norm and of the 4-bit floats, pinned without a GPU: hand-worked
values, exhaustive rounding against brute force, the formula's gradient against
central differences."""
import itertools

import numpy as np
import pytest

from oracle import layer_oracle as O


def test_e2m1_every_midpoint_goes_to_the_even_code():
    mids = (O.E2M1[:-1] + O.E2M1[1:]) / 2
    assert list(O.e2m1(mids)) == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]
    assert list(O.e2m1(-mids)) == [-0.0, -1.0, -1.0, -2.0, -2.0, -4.0, -4.0]
    eps = 1e-9
    assert list(O.e2m1(mids + eps)) == list(O.E2M1[1:])
    assert list(O.e2m1(mids - eps)) == list(O.E2M1[:-1])
    assert list(O.e2m1(np.array([5.0, 7.9, 1e30, -6.5]))) == [4.0, 6.0, 6.0, -6.0]


def test_e4m3_table_and_rounding():
    assert O.E4M3[-1] == 448.0 and O.E4M3[1] == 2.0 ** -9 and O.E4M3[8] == 2.0 ** -6 and len(O.E4M3) == 127
    assert (O.e4m3(O.E4M3) == O.E4M3).all()
    mids = (O.E4M3[:-1] + O.E4M3[1:]) / 2
    want = np.array([O.E4M3[i] if i % 2 == 0 else O.E4M3[i + 1] for i in range(126)])
    assert (O.e4m3(mids) == want).all()
    assert O.e4m3(np.array([500.0]))[0] == 448.0


def test_block32_scale_is_the_power_of_two_below_the_maximum():
    x = np.zeros((1, 64), np.float32)
    x[0, :4] = [6.0, -3.0, 0.25, 0.75]        # maximum 6: scale 1
    x[0, 32:35] = [7.5, 1.0, 0.3]             # still scale 1: 7.5 is cut to 6
    v, g = O.fp4(x, 32)
    assert list(v[0, :4]) == [6.0, -3.0, 0.0, 1.0] and list(v[0, 32:35]) == [6.0, 1.0, 0.5] and g[0] == 1.0
    x[0, 0] = 8.0                             # scale 2
    assert list(O.fp4(x, 32)[0][0, :4]) == [8.0, -3.0, 0.0, 1.0]
    tiny = np.full((1, 32), 2.0 ** -130, np.float32)   # below the smallest scale's codes: 2^-127 * (1/8) -> 0
    assert (O.fp4(tiny, 32)[0] == 0).all()
    tiny[0, 0] = 2.0 ** -126
    assert O.fp4(tiny, 32)[0][0, 0] == 2.0 ** -126


def test_block16_full_scale_and_row_scale():
    x = np.zeros((2, 32), np.float32)
    x[0, 0], x[0, 16] = 2688.0, 6.0           # g = 1 (to float32 rounding), scales 448 and 1
    x[0, 17:20] = [3.0, -1.4, 0.2]
    v, g = O.fp4(x, 16)
    assert abs(g[0] - 1.0) < 1e-6 and g[1] == 1.0
    assert v[0, 0] == 2688.0 and list(v[0, 16:20]) == [6.0, 3.0, -1.5, 0.0]
    assert (v[1] == 0).all()
    # the values stand for x within half a step of e2m1 and of e4m3
    r = np.random.default_rng(0).standard_normal((7, 100)).astype(np.float32)
    v, g = O.fp4(r, 16)
    b = np.abs(np.pad(r, ((0, 0), (0, 12))).reshape(7, -1, 16)).max(axis=2).repeat(16, axis=1)[:, :100]
    assert (np.abs(v * g[:, None] - r) <= b * (1 / 6 + 1 / 16) + 1e-6).all()


def test_nan_and_infinity_poison_their_block_or_row():
    x = np.ones((3, 64), np.float32)
    x[0, 40], x[1, 3] = np.inf, np.nan
    v, g = O.fp4(x, 32)
    assert np.isnan(v[0, 32:]).all() and (v[0, :32] == 1).all() and np.isnan(v[1, :32]).all() and (v[2] == 1).all()
    v, g = O.fp4(x, 16)
    assert np.isnan(g[:2]).all() and g[2] > 0


def test_product_against_brute_force():
    rng = np.random.default_rng(3)
    a, b = rng.standard_normal((3, 40)).astype(np.float32), rng.standard_normal((4, 40)).astype(np.float32)
    for block in (16, 32):
        y, mag = O.fp4_matmul(a, b, block)
        va, ga = O.fp4(a, block)
        vb, gb = O.fp4(b, block)
        for m, n in itertools.product(range(3), range(4)):
            s = sum(va[m, k] * vb[n, k] for k in range(40)) * ga[m] * gb[n]
            assert abs(s - y[m, n]) <= 1e-12 * mag[m, n]


def test_norm_hand_worked_and_within_half_a_step():
    x = np.array([[3.0, -4.0, 0.0, 0.0]], np.float32)
    w = np.array([1.0, 1.0, 5.0, 1.0], np.float32)
    q, s, h, r = O.rms_norm_s8(x, w, None, 0.0, False)
    assert list(q[0]) == [95, -127, 0, 0] and abs(r[0] - 0.4) < 1e-12 and abs(s[0] - 4 * 0.4 / 127) < 1e-9
    rng = np.random.default_rng(1)
    x, w = rng.standard_normal((9, 50)).astype(np.float32), rng.standard_normal(50).astype(np.float32)
    q, s, h, r = O.rms_norm_s8(x, w, rng.standard_normal((9, 50)).astype(np.float32), 1e-6, True)
    assert (np.abs(q * s[:, None] - O.rms_norm(h, w, 1e-6)) <= s[:, None] * 0.50001).all()
    q, s, _, _ = O.rms_norm_s8(np.zeros((1, 3), np.float32), w[:3], None, 1e-6, False)
    assert (q == 0).all() and s[0] == 1.0
    q, s, _, _ = O.rms_norm_s8(np.array([[1, np.inf, 0]], np.float32), w[:3], None, 1e-6, False)
    assert (q == 0).all() and np.isnan(s[0])


@pytest.mark.parametrize("H", [1, 2, 33])
def test_norm_gradient_against_central_differences(H):
    rng = np.random.default_rng(H)
    h, w = rng.standard_normal((4, H)), rng.standard_normal(H)
    dy, dh = rng.standard_normal((4, H)), rng.standard_normal((4, H))
    eps = 1e-6
    rstd = 1 / np.sqrt((h ** 2).mean(axis=1) + eps)
    dx, dw = O.rms_norm_backward(dy, h, w, rstd, dh)

    def loss(hh, ww):
        return (O.rms_norm(hh, ww, eps) * dy).sum() + (hh * dh).sum()
    t = 1e-6
    for i, j in itertools.product(range(4), range(H)):
        d = np.zeros_like(h)
        d[i, j] = t
        assert abs((loss(h + d, w) - loss(h - d, w)) / (2 * t) - dx[i, j]) < 1e-6 * (1 + abs(dx).max())
    for j in range(H):
        d = np.zeros_like(w)
        d[j] = t
        assert abs((loss(h, w + d) - loss(h, w - d)) / (2 * t) - dw[j]) < 1e-6 * (1 + abs(dw).max())


def test_bf16_rounding_ties_to_even():
    x = np.array([1.0 + 2.0 ** -8, 1.0 + 3 * 2.0 ** -8, 1.0 + 2.0 ** -8 + 2.0 ** -20], np.float32)
    assert list(O.bf16_round(x)) == [1.0, 1.0 + 2.0 ** -6, 1.0 + 2.0 ** -7]
