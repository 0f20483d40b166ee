"""CPU pins of the microscaling and clip oracle: the definition by brute force,
the format's layout, and planted mistakes that each fail a pin."""
import math

import numpy as np
import pytest

from oracle import microscaling as MX


@pytest.mark.parametrize("amax", [6.0, 6.0000001, 5.9, 3.0, 3.0000001, 1e-30, 1e-45, 1.0, 448.0, 3.4e38, 0.0])
def test_block_exponent_is_the_smallest_sufficient(amax):
    amax = float(np.float32(amax))
    k = MX.block_exponent(amax)
    assert k >= -127 and amax <= 6.0 * 2.0 ** k
    if k > -127:
        assert amax > 6.0 * 2.0 ** (k - 1)


def test_nearest_against_brute_force():
    g = np.random.default_rng(1)
    x = g.standard_normal((3, 75)) * np.exp(3 * g.standard_normal((3, 1)))
    codes, scales = MX.quantize(x)
    v = MX.values(codes, scales, 75)
    for i in range(3):
        for j in range(75):
            unit = 2.0 ** (int(scales[i, j // 32]) - 127)
            best = min(abs(abs(x[i, j]) - q * unit) for q in MX.GRID)
            assert abs(abs(v[i, j]) - abs(x[i, j])) == pytest.approx(best, abs=1e-300)
            assert v[i, j] == 0 or np.sign(v[i, j]) == np.sign(x[i, j])


def test_ties_go_to_the_even_code():
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    want = [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]
    x = np.array([ties + [6.0] + [-t for t in ties]])
    assert MX.round_values(x)[0].tolist() == want + [6.0] + [-w for w in want]


def test_stochastic_rounding_is_unbiased_over_the_bytes():
    # over all 256 bytes the mean is within half a byte's step of the value
    x = np.array([[6.0, 0.1, 0.3, 0.74, 1.1, 1.9, 2.3, 3.7, 4.2, 5.9, -2.3]])
    total = np.zeros(x.shape)
    for r in range(256):
        total += MX.round_values(x, np.full(x.shape, r, np.uint8))
    gap = np.array([0, .5, .5, .5, .5, .5, 1, 1, 2, 2, 1])
    assert np.all(np.abs(total / 256 - x) <= gap / 512 + 1e-15)


def test_exact_values_are_never_moved():
    x = np.array([[0.5, -1.5, 6.0, 0.0, 3.0, 4.0]]) * 2.0 ** -20
    for r in (0, 255):
        assert np.array_equal(MX.round_values(x, np.full(x.shape, r, np.uint8)), x)
    assert np.array_equal(MX.round_values(x), x)


def test_non_finite_blocks():
    x = np.ones((1, 70))
    x[0, 3], x[0, 65] = np.inf, np.nan
    codes, scales = MX.quantize(x)
    assert scales[0].tolist()[0] == 255 and scales[0, 2] == 255 and scales[0, 1] != 255
    v = MX.values(codes, scales, 70)
    assert np.isnan(v[0, :32]).all() and np.isnan(v[0, 64:]).all() and (v[0, 32:64] == 1).all()


def test_scale_tiles_are_a_bijection():
    rows, cols = 70, 600
    nb = -(-cols // 32)
    seen = {MX.scale_index(i, b, cols) for i in range(rows) for b in range(nb)}
    assert len(seen) == rows * nb and max(seen) < 3 * 3 * 256
    # rows i and i + 16 and two neighbouring blocks make one aligned dword
    for i in (0, 9, 47):
        for b in (0, 2, 4, 14):
            j = [MX.scale_index(i + h, b + s, cols) for h in (0, 16) for s in (0, 1)]
            assert j[0] % 4 == 0 and j == list(range(j[0], j[0] + 4))


def test_packing_is_low_nibble_first():
    c = np.arange(32, dtype=np.uint8)[None, :] % 16
    assert MX.pack_codes(c)[0, 0] == 0x10 and MX.pack_codes(c)[0, 3] == 0x76


def test_clip_closed_form():
    norm, c, per, outs = MX.clip([np.array([3.0]), np.array([0.0, 4.0])], 2.5)
    assert norm == 5.0 and per == [3.0, 4.0] and c == pytest.approx(0.5, rel=1e-6)
    assert outs[1][1] == pytest.approx(2.0, rel=1e-6)
    assert MX.clip([np.array([3.0])], 7.0)[1] == 1.0
    assert MX.clip([np.array([3.0])], 1.0, scale=-2.0)[0] == 6.0
    assert math.isnan(MX.clip([np.array([np.nan, 1.0])], 1.0)[1])
    assert MX.clip([np.array([np.inf, 1.0])], 1.0)[1] == 0.0


def test_planted_mistakes_fail_a_pin():
    g = np.random.default_rng(2)
    x = g.standard_normal((2, 64))
    good = MX.round_values(x)
    # a scale from floor(log2 max) - 2 saturates values above 6 units
    k = np.floor(np.log2(np.abs(x[0, :32]).max())) - 2
    assert np.abs(x[0, :32]).max() > 6.0 * 2.0 ** k or not np.array_equal(
        np.clip(x[0, :32], -6 * 2.0 ** k, 6 * 2.0 ** k), good[0, :32])
    # blocks along the other axis
    assert not np.array_equal(MX.round_values(x.T).T, good)
    # swapped nibbles
    c, _ = MX.quantize(x)
    assert not np.array_equal((c[:, 1::2] | (c[:, 0::2] << 4)), MX.pack_codes(c))


def test_infinite_limit_clips_nothing():
    norm, c, _, outs = MX.clip([np.array([np.inf, 2.0])], math.inf)
    assert norm == math.inf and c == 1.0 and outs[0].tolist() == [math.inf, 2.0]
    assert MX.clip([np.array([3.0])], math.inf)[1] == 1.0
    assert math.isnan(MX.clip([np.array([np.nan, np.inf])], math.inf)[1])
