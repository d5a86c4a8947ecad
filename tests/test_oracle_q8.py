"""Pins of the 8-bit row oracle: codes and scales against exact rationals,
the norm's gradient against central differences."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import q8_oracle as Q


def _round_half_even(f: Fraction) -> int:
    n = f.numerator // f.denominator
    rest = f - n
    if rest > Fraction(1, 2) or (rest == Fraction(1, 2) and n % 2):
        n += 1
    return n


@pytest.mark.parametrize("kind", ["f32", "bf16", "ties"])
def test_codes_and_scale_against_rationals(kind):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((12, 40)).astype(np.float32)
    if kind == "bf16":
        x = (x.view(np.uint32) & 0xFFFF0000).view(np.float32)
    if kind == "ties":
        # largest magnitude a; entries a (2 n + 1) / 254 are exact ties when representable
        for m in range(12):
            a = np.float32(127 * 2.0 ** (m - 6))
            x[m] = ((2 * rng.integers(-127, 127, 40) + 1) * np.float32(2.0 ** (m - 7))).astype(np.float32)
            x[m, 3] = -a
    codes, scale = Q.quantize_rows(x)
    for m in range(x.shape[0]):
        a = max(abs(Fraction(float(v))) for v in x[m])
        assert Fraction(float(scale[m])) == Fraction(float(np.float32(float(a)) / np.float32(127)))
        for k in range(x.shape[1]):
            assert codes[m, k] == _round_half_even(127 * Fraction(float(x[m, k])) / a)


def test_special_rows():
    x = np.array([[0, 0, 0], [np.inf, 1, 2], [1, np.nan, 2], [1, -2, 0.5]], np.float32)
    codes, scale = Q.quantize_rows(x)
    assert (codes[:3] == 0).all() and scale[0] == 0 and np.isnan(scale[1]) and np.isnan(scale[2])
    assert list(codes[3]) == [64, -127, 32]  # 63.5 and 31.75


def test_rmsnorm_gradient_against_differences():
    rng = np.random.default_rng(1)
    M, d, eps = 3, 7, 1e-3
    x, res, dy, dh = (rng.standard_normal((M, d)) for _ in range(4))
    gamma = 1 + 0.3 * rng.standard_normal(d)
    h, rstd, _ = Q.rmsnorm(x, gamma, eps, res)
    dx, dgamma = Q.rmsnorm_backward(h, gamma, rstd, dy, dh)

    def value(x, gamma):
        h, _, y = Q.rmsnorm(x, gamma, eps, res)
        return (dy * y).sum() + (dh * h).sum()

    t = 1e-6
    for m in range(M):
        for k in range(d):
            e = np.zeros((M, d)); e[m, k] = t
            assert abs((value(x + e, gamma) - value(x - e, gamma)) / (2 * t) - dx[m, k]) < 1e-7
    for k in range(d):
        e = np.zeros(d); e[k] = t
        assert abs((value(x, gamma + e) - value(x, gamma - e)) / (2 * t) - dgamma[k]) < 1e-7
