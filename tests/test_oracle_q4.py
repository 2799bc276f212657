"""The 4-bit cache's reference, held to blocks worked out by hand and to what follows from the definition."""
import numpy as np
import pytest

from oracle import paged_q4 as q4


def one(x, rest=0.0):
    b = np.full(32, rest)
    b[: len(x)] = x
    codes, byte = q4.block(b)
    return codes[: len(x)].tolist(), byte


def test_by_hand():
    # 6 is the largest magnitude: power 1, so the values are the numbers themselves
    assert one([6.0, -0.5, 1.5, 3.0, 0.2, -4.9]) == ([7, 9, 3, 5, 0, 14], 127)
    # 7 passes 6: power 2; 7 / 2 = 3.5 lies between 3 (code 5) and 4 (code 6): the even one
    assert one([7.0, 1.0, 5.0]) == ([6, 1, 4], 128)
    # halves between neighbours, at power 1 (the block holds a 6)
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    assert one(ties + [6.0])[0] == [0, 2, 2, 4, 4, 6, 6, 7]
    assert one([-t for t in ties] + [6.0])[0] == [8, 10, 10, 12, 12, 14, 14, 7]
    assert one([0.0]) == ([0], 1)


def test_edges_of_the_powers():
    assert one([6 * 2.0 ** -126])[1] == 1 and one([2.0 ** -140])[1] == 1
    assert one([6 * 2.0 ** 125]) == ([7], 252)
    assert one([np.finfo(np.float32).max]) == ([7], 252)   # held down to 6 * 2^125
    for e in (-100, -1, 0, 1, 60):
        assert one([6 * 2.0 ** e])[1] == e + 127
        assert one([np.nextafter(np.float32(6 * 2.0 ** e), np.float32(np.inf))])[1] == e + 128


@pytest.mark.parametrize("odd", [np.inf, -np.inf, np.nan])
def test_not_finite(odd):
    codes, byte = q4.block([1.0, odd] + [0.0] * 30)
    assert byte == 255 and (codes == 0).all()
    assert np.isnan(q4.values(np.zeros(16, np.uint8), np.array([255]))).all()


def test_error_and_idempotence():
    x = np.random.default_rng(5).standard_normal((40, 96)) * np.exp(np.random.default_rng(6).standard_normal((40, 1)) * 20)
    codes, scales = q4.quantise(x)
    y = q4.values(codes, scales)
    power = 2.0 ** (scales.astype(float) - 127)
    err = np.abs(y - x).reshape(40, 3, 32) / power[..., None]
    top = np.abs(x).reshape(40, 3, 32).max(-1)
    assert (top <= 6 * power).all() and (top > 3 * power).all()
    assert (err <= 1.0).all()   # half of the widest gap, 4 to 6
    again = q4.quantise(y)
    assert (q4.values(*again) == y).all()
    # the nearest value, and none nearer
    grid = np.concatenate([q4.VALUES, -q4.VALUES])
    best = np.abs(x.reshape(40, 3, 32, 1) / power[..., None, None] - grid).min(-1)
    np.testing.assert_allclose(err, best, atol=1e-12)


def test_packing():
    x = np.zeros(64)
    x[0], x[1], x[33] = 1.0, 6.0, -3.0
    codes, scales = q4.quantise(x)
    # the first block at power 1; the second's 3 is 6 at power 1/2
    assert codes[0] == 0x72 and codes[16] == 0xF0 and scales.tolist() == [127, 126]
    assert codes.shape == (32,) and (q4.values(codes, scales) == x).all()
