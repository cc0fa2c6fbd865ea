"""Pins of the microscaled 4-bit oracle and of its Python binding's host
checks (no GPU): rounding, ties, saturation, scales at the ends of the range,
packing order, short last blocks."""
import math

import numpy as np
import pytest

from oracle import mxfp4 as M


def test_ties_and_saturation():
    # between neighbours 0 .5 1 1.5 2 3 4 6: a tie goes to the even index (0, 1, 2, 4)
    for a, want in ((0.25, 0.0), (0.75, 1.0), (1.25, 1.0), (1.75, 2.0), (2.5, 2.0), (3.5, 4.0), (5.0, 4.0), (5.01, 6.0),
                    (7.99, 6.0), (100.0, 6.0), (0.26, 0.5), (0.0, 0.0)):
        assert M.MAGNITUDES[M.element(a)] == want, a


def test_block_by_hand():
    W = np.zeros((1, 33))
    W[0, :5] = [4.0, -3.0, 0.5, -0.25, 7.9]          # m = 7.9: e = 0
    W[0, 32] = 0.4                                    # short second block: floor(log2 .4) - 2 = -4: .4 / 2^-4 = 6.4 -> 6
    codes, scales = M.quantize(W)
    assert codes.shape == (1, 32) and scales.shape == (1, 16)
    assert list(scales[0, :2]) == [127, 123] and not scales[0, 2:].any()
    assert list(codes[0, :3]) == [6 | (13 << 4), 1 | (8 << 4), 7]
    assert codes[0, 16] == 7 and not codes[0, 17:].any()
    val = M.dequantize(codes, scales, 33)
    assert list(val[0, :5]) == [4.0, -3.0, 0.5, 0.0, 6.0] and val[0, 32] == 6 * 2.0 ** -4


def test_range_ends():
    for m, code in ((0.0, 0), (2.0 ** -149, 0), (2.0 ** -126, 0), (2.0 ** -125, 0), (2.0 ** -124, 1), (1.0, 125),
                    (2.0 ** 127, 252), (float(np.finfo(np.float32).max), 252), (math.inf, 255), (math.nan, 255)):
        _, scales = M.quantize(np.array([[m]]))
        assert scales[0, 0] == code, m
    codes, scales = M.quantize(np.array([[1.0] * 31 + [math.nan] + [1.0]]))
    assert not codes[0, :16].any() and scales[0, 0] == 255
    val = M.dequantize(codes, scales, 33)
    assert np.isnan(val[0, :32]).all() and val[0, 32] == 1.0


def test_elements_agree_with_scalar_rule():
    rng = np.random.default_rng(3)
    W = rng.standard_normal((3, 64)) * np.exp(rng.standard_normal((3, 64)))
    codes, scales = M.quantize(W)
    for n in range(3):
        for j in range(64):
            e = int(scales[n, j // 32]) - 127
            nib = (codes[n, j // 2] >> (4 * (j % 2))) & 15
            assert nib & 7 == M.element(abs(W[n, j]) / 2.0 ** e) and (nib >> 3) == (W[n, j] < 0)


@pytest.mark.parametrize("d", [1, 31, 32, 33, 511, 512, 513, 4096])
def test_values_requantise_to_themselves(d):
    """Every value of a block lies on its grid; a second pass gives the same values (its scale may be one lower
    where rounding took the largest element down)."""
    rng = np.random.default_rng(d)
    val = M.dequantize(*M.quantize(rng.standard_normal((4, d))), d)
    assert np.array_equal(M.dequantize(*M.quantize(val), d), val)
