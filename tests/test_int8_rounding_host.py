"""The 8-bit rounding by one multiply with a rounded-up reciprocal is rint of the
exact quotient: the argument beside the kernel, in whole numbers."""
import numpy as np
import pytest


def reciprocal_up(M):
    """127 / M rounded up to fp32, as a whole number of 2^-40."""
    r = np.float32(np.float64(127) / np.float64(M))
    if int(np.float64(r) * 2.0 ** 40) * M < 127 << 40:
        r = np.nextafter(r, np.float32(np.inf))
    got = int(np.float64(r) * 2.0 ** 40)                  # (exact: 24 bits above 2^-25)
    assert np.float64(r) * 2.0 ** 40 == got and got * M >= 127 << 40
    return got


def rint_of(num, shift):
    """Whole numbers num / 2^shift to the nearest, ties to even."""
    q, rest, half = num >> shift, num & ((1 << shift) - 1), 1 << (shift - 1)
    return q + ((rest > half) | ((rest == half) & (q & 1 == 1)))


@pytest.mark.parametrize("s", range(10))
def test_rounding(s):
    A = np.arange(0, 256, dtype=np.int64)                 # (below 128: denormals)
    for M in range(1, 256):
        a = A[A <= M << s]
        # the exact quotient 127 a / (M 2^s): twice its distance to the tie above its floor, over M 2^s
        den = M << s
        q, rest = np.divmod(127 * a, den)
        tie = 2 * rest - den                              # 0 at a tie
        want = q + ((tie > 0) | ((tie == 0) & (q & 1 == 1)))
        up = reciprocal_up(M)
        # the distance |tie| / (2 M 2^s) of what is no tie is over 128 times the error
        # a (up 2^-40 - 127 / M) 2^-s, both sides times 2 M 2^s 2^40
        error = 2 * a * (up * M - (127 << 40))
        assert (128 * error[tie != 0] < np.abs(tie[tie != 0]) << 40).all()
        assert (rint_of(a * up, 40 + s) == want).all()


def test_the_nearest_that_is_no_tie():
    """Far below the top of the range a quotient may come closer to a tie than any fixed distance."""
    assert abs(127 * 255 / (253 * 2 ** 8) - 0.5) == pytest.approx(1 / 64768)
