"""Pins of the serving oracle: quantised rows by hand and by exact rational
arithmetic, and the expert layer against its steps' own definitions."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import experts as OE


def test_quantize_by_hand():
    x = np.array([[0.0, 0.0, 0.0], [127.0, -1.0, 0.5], [-254.0, 3.0, 5.0], [63.5, 0.25, -0.75]])
    q, s = OE.quantize(x)
    assert s.tolist() == [0.0, 1.0, 2.0, 0.5]
    # ties go to the even integer: 0.5 -> 0, 1.5 -> 2, 2.5 -> 2, 0.5 -> 0, -1.5 -> -2
    assert q.tolist() == [[0, 0, 0], [127, -1, 0], [-127, 2, 2], [127, 0, -2]]


def _nearest(x, s):
    v = Fraction(x) / Fraction(s)
    lo = v.numerator // v.denominator
    d = v - lo
    n = lo if d < Fraction(1, 2) or (d == Fraction(1, 2) and lo % 2 == 0) else lo + 1
    return max(-127, min(127, n))


@pytest.mark.parametrize("size", [1.0, 1e-30, 1e30, 2.0 ** -146])
def test_quantize_against_rationals(size):
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((40, 9)) * size).astype(np.float32)
    x[:, 1] = x[:, 0] / 2  # quotients near a tie
    q, s = OE.quantize(x.astype(np.float64))
    for i in range(len(x)):
        m = Fraction(float(np.abs(x[i]).max())) / 127
        # the float32 nearest to the exact quotient
        for other in (np.nextafter(s[i], np.float32(0)), np.nextafter(s[i], np.float32(np.inf))):
            assert abs(Fraction(float(s[i])) - m) <= abs(Fraction(float(other)) - m)
        if s[i]:
            assert [_nearest(float(v), float(s[i])) for v in x[i]] == q[i].tolist()


@pytest.mark.parametrize("name", OE.ACTIVATIONS)
def test_decode_against_the_steps(name):
    """The layer as dispatch, the grouped products and combine make it."""
    rng = np.random.default_rng(6)
    T, k, E, h, f = 5, 3, 4, 6, 7
    x = rng.standard_normal((T, h))
    wg, wu, wd = rng.standard_normal((E, f, h)), rng.standard_normal((E, f, h)), rng.standard_normal((E, h, f))
    idx = rng.integers(0, E, (T, k))
    w = rng.random((T, k))
    order = np.argsort(idx.reshape(-1), kind="stable")
    off = np.concatenate([[0], np.cumsum(np.bincount(idx.reshape(-1), minlength=E))])
    rows = x[order // k]
    z = OE.linear(OE.gated(rows, off, wg, wu, name)[0], off, wd)[0]
    want = np.zeros_like(x)
    np.add.at(want, order // k, w.reshape(-1)[order][:, None] * z)
    got, parts = OE.decode(x, idx, w, wg, wu, wd, name)
    assert np.allclose(got, want, rtol=1e-12, atol=1e-12)
    assert len(parts) == T * k


def test_decode_passes_over_absent_experts():
    x = np.ones((2, 2))
    one = np.ones((1, 2, 2))
    y, parts = OE.decode(x, np.array([[0, -1], [1, 7]]), np.full((2, 2), 0.5), one, one, one, "none")
    assert y.tolist() == [[4.0, 4.0], [0.0, 0.0]] and list(parts) == [(0, 0)]
