"""Pins of the MX4 oracle: hand-worked codes and scales, brute-force rounding,
round trips, closed forms of the product, the layer and the norms."""
import itertools
import types

import numpy as np
import pytest

from oracle import mx4


def block(first):
    v = np.zeros(32)
    v[:len(first)] = first
    return v


@pytest.mark.parametrize("vals,byte,codes", [
    ([6, -6, 0.5, 3], 127, [0xF7, 0x51]),                # scale 1
    ([7.9, 1], 127, [0x27]),                             # above 6: saturates
    ([8, 1], 128, [0x16]),                               # amax 8: scale 2, 1/2 = 0.5
    ([0.25, 4], 127, [0x60]),                            # tie 0.25 -> 0
    ([0.75, 4], 127, [0x62]),                            # tie 0.75 -> 1
    ([1.25, 4, 1.75, 2.5, 3.5, 5.0], 127, [0x62, 0x44, 0x66]),
    ([-0.1, 4], 127, [0x68]),                            # rounds to minus zero
    ([2.0 ** -126], 0, [0x04]),                          # 2**-126 / 2**-127
    ([2.0 ** -149], 0, [0x00]),
])
def test_hand_worked_blocks(vals, byte, codes):
    c, b = mx4.quantize(block(vals))
    assert b.tolist() == [byte]
    assert c[:len(codes)].tolist() == codes and not c[len(codes):].any()


def test_zero_and_non_finite_blocks():
    c, b = mx4.quantize(np.zeros(32))
    assert b[0] == 0 and not c.any()
    for bad in (np.nan, np.inf, -np.inf):
        c, b = mx4.quantize(np.concatenate([block([1, bad]), block([4.0])]))
        assert b.tolist() == [255, 127] and not c[:16].any() and c[16] == 6
        v = mx4.values(c, b)
        assert np.isnan(v[:32]).all() and v[32] == 4


def test_rounding_is_nearest_with_even_ties():
    a = np.arange(0, 8.001, 1 / 64)
    for v, code in zip(a, mx4.round_codes(a)):
        d = np.abs(mx4.MAGNITUDES - v)
        best = [i for i in range(8) if d[i] == d.min()]
        assert code == (best[0] if len(best) == 1 else next(i for i in best if i % 2 == 0))


def test_round_trip_of_all_bytes():
    codes = np.arange(256, dtype=np.uint8).reshape(16, 16)
    codes[:, 0] = 0x77                                    # a 6 in every block keeps its scale
    scales = np.full((16, 1), 120, np.uint8)
    c, b = mx4.quantize(mx4.values(codes, scales))
    assert np.array_equal(c, codes) and np.array_equal(b, scales)


def test_quantisation_error_is_at_most_a_sixth_of_the_largest():
    x = np.random.default_rng(3).standard_normal((50, 64))
    v = mx4.values(*mx4.quantize(x)).reshape(50, 2, 32)
    xb = x.reshape(50, 2, 32)
    # amax in [4, 8) scale units: half a step of the coarsest interval is 1 unit, saturation costs less than 2
    assert (np.abs(v - xb).max(-1) <= np.abs(xb).max(-1) / 4).all()


def test_product_closed_form_and_groups():
    w = np.zeros((2, 3, 64))
    w[0, 1, 5], w[1, 2, 40] = 2.0, -3.0
    x = np.arange(4 * 64, dtype=np.float64).reshape(4, 64)
    y, mag = mx4.product(x, w, [0, 1, 4])
    expect = np.zeros((4, 3))
    expect[0, 1] = 2 * x[0, 5]
    expect[1:, 2] = -3 * x[1:, 40]
    assert np.array_equal(y, expect) and np.array_equal(mag, np.abs(expect))


def test_layer_is_the_weighted_sum_of_its_experts():
    shape = types.SimpleNamespace(hidden=64, n_experts=3, n_shared=1)
    rng = np.random.default_rng(5)
    mats = [[mx4.values(*mx4.quantize(rng.standard_normal(s))) for s in ((32, 64), (32, 64), (64, 32))] for _ in range(4)]
    x = rng.standard_normal((5, 64))
    idx = np.array([[0, 2], [1, 1], [-1, 2], [-1, -1], [2, 0]])
    w = rng.random((5, 2)).astype(np.float32)
    y, bound = mx4.layer(shape, lambda e: mats[e], lambda s: mats[3], x, idx, w)
    xv = mx4.values(*mx4.quantize(x))
    for t in range(5):
        ref = np.zeros(64)
        for m, c in [(mats[i], w[t, j]) for j, i in enumerate(idx[t]) if i >= 0] + [(mats[3], 1.0)]:
            g, u = m[0] @ xv[t], m[1] @ xv[t]
            ref += c * (m[2] @ mx4.values(*mx4.quantize(g / (1 + np.exp(-g)) * u)))
        assert np.allclose(y[t], ref, rtol=1e-12, atol=1e-12)
    assert (bound > 0).all() and (bound < 0.5 * np.abs(y).max()).all()


def test_reach_covers_every_perturbation():
    rng = np.random.default_rng(7)
    h = rng.standard_normal((20, 32))
    h[:, 0] = 4.0 * (1 + 1e-4 * rng.standard_normal(20))     # the block's largest near a power of two
    err = 2e-4 * np.abs(h)
    v0, reach = mx4._quant_reach(h, err)
    for _ in range(20):
        v = mx4.values(*mx4.quantize(h + err * rng.uniform(-1, 1, h.shape)))
        assert (np.abs(v - v0) <= reach + 1e-12).all()
    assert reach.any()


@pytest.mark.parametrize("post,gate,pre", list(itertools.product([False, True], repeat=3)))
def test_block_norm_closed_form(post, gate, pre):
    # constant rows: rms(c) = sign(c), so every step has a value by hand
    x, y = np.full((2, 8), 3.0), np.full((2, 8), -2.0)
    n = 8
    xo, no = mx4.block_norm(x, y, np.full(n, 5.0) if post else None, np.full(n, 0.5) if gate else None, 0.25,
                            np.full(n, 4.0) if pre else None, eps=0.0)
    r = (-5.0 if post else -2.0) * (0.5 if gate else 1.0)
    assert np.allclose(xo, 3.0 + 0.25 * r, rtol=1e-14)
    assert np.allclose(no, np.sign(3.0 + 0.25 * r) * (4.0 if pre else 1.0), rtol=1e-14)
