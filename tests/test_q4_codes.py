"""The codes of q4 rows are rounded right although the kernel multiplies by an
approximate reciprocal of the scale: its steps (one product, one remainder, one
correction, all rounded to f32) give, for any reciprocal within two units of the
last place, a quotient on the same side of every middle between two codes as the
true one, and on the middle exactly where that is."""
import numpy as np
import pytest

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
MIDDLES = (LEVELS[1:] + LEVELS[:-1]) / 2
AROUND = 20000             # floats on either side of a middle
f32, f64 = np.float32, np.float64


def _rounded_sum(p, b):
    """p + b, two f64 numbers, rounded once to f32 (their sum may not be an f64 number:
    a tie in its f64 rounding is settled by what that left)."""
    hi = p + b
    t = hi - p
    lo = (p - (hi - t)) + (b - t)          # exactly what hi is short of (Knuth)
    c = hi.astype(f32)
    back = c.astype(f64)
    other = np.nextafter(c, np.where(hi > back, f32(np.inf), f32(-np.inf)).astype(f32))
    tie = (hi != back) & (np.abs(hi - back) == np.abs(other.astype(f64) - hi))
    up = np.maximum(c, other)
    down = np.minimum(c, other)
    return np.where(tie & (lo > 0), up, np.where(tie & (lo < 0), down, c))


def _quotients(a, s, r):
    """The kernel's steps for numerators a (f32), a scale s and its reciprocal r."""
    b = (a.astype(f64) * f64(r)).astype(f32)               # 48 bits: exact before the rounding
    e = (a.astype(f64) - f64(s) * b.astype(f64)).astype(f32)   # exact as well
    return _rounded_sum(e.astype(f64) * f64(r), b.astype(f64))


@pytest.mark.parametrize("fraction", range(8))
def test_quotients_fall_on_the_right_side_of_every_middle(fraction):
    s = f32(1 + fraction / 8)
    for off in (-2, -1, 0, 1, 2):
        r = f32(1 / f64(s))
        for _ in range(abs(off)):
            r = np.nextafter(r, f32(np.inf if off > 0 else 0))
        for m in MIDDLES:
            at = f32(m * f64(s))
            assert f64(at) == m * f64(s)                       # a middle times a scale is a float
            a = (at.view(np.int32) + np.arange(-AROUND, AROUND + 1, dtype=np.int32)).astype(np.int32).view(f32)
            q = _quotients(a, s, r).astype(f64)
            assert np.array_equal(np.sign(q - m), np.sign(a.astype(f64) - f64(at))), (off, m)


def test_the_sum_is_rounded_once():
    """Against whole numbers, at sums whose f64 rounding is a tie of f32."""
    b = f64(1.0)
    for p, want in ((2.0 ** -24, 1.0), (2.0 ** -24 + 2.0 ** -60, 1 + 2.0 ** -23), (2.0 ** -24 - 2.0 ** -60, 1.0),
                    (3 * 2.0 ** -24, 1 + 2.0 ** -22), (3 * 2.0 ** -24 - 2.0 ** -60, 1 + 2.0 ** -23), (-2.0 ** -25, 1.0),
                    (-2.0 ** -25 - 2.0 ** -70, 1 - 2.0 ** -24)):
        assert f64(_rounded_sum(np.array([p]), np.array([b]))[0]) == want, p
