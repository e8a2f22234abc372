"""The MXFP4 oracle against closed forms."""
import numpy as np

from oracle import mx4


def _block(*head):
    return np.array(list(head) + [0.0] * (32 - len(head)))


def test_ties_go_to_the_even_code():
    # amax 6 makes the scale 1; midpoints between neighbouring values
    v = _block(6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0)
    c, s = mx4.quantize(v)
    assert s.tolist() == [127]
    got = mx4.dequantize(c, s)[:10]
    assert got.tolist() == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 0.0, -4.0]


def test_scale_is_the_power_below_the_largest_over_four():
    for top, byte in ((4.0, 127), (7.99, 127), (8.0, 128), (3.99, 126), (1.0, 125), (0.0, 127),
                      (2.0 ** -130, 0), (2.0 ** 127, 252), (np.inf, 255), (np.nan, 255)):
        c, s = mx4.quantize(_block(top, top / 2 if np.isfinite(top) else 1.0))
        assert s.tolist() == [byte], top
        if byte == 255:
            assert not c.any() and np.isnan(mx4.dequantize(c, s)).all()


def test_every_value_survives_a_round_trip():
    for e in (-120, -3, 0, 5, 100):
        v = np.concatenate([mx4.VALUES, -mx4.VALUES, mx4.VALUES, mx4.VALUES[::-1]]) * 2.0 ** e
        c, s = mx4.quantize(v)
        assert np.array_equal(mx4.dequantize(c, s), v)


def test_error_bound():
    # under 7 (in units of the scale) the step is at most 2, so the error at most 1; from 7 to 8
    # the value saturates at 6
    v = np.random.default_rng(0).normal(size=(64, 256)) * np.exp(np.linspace(-9, 9, 64))[:, None]
    c, s = mx4.quantize(v)
    unit = np.repeat(np.exp2(s.astype(np.float64) - 127), 32, -1)
    err = np.abs(mx4.dequantize(c, s) - v) / unit
    assert err.max() <= 2.0 and err[np.abs(v) / unit <= 7].max() <= 1.0
