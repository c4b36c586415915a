"""The few-row kernel's splits of the probabilities and of Q over an 8-bit cache, restated in fp64 with the formats' own roundings, against
the errors that fa.h and the kernel state for them.

P is rounded to fp16 and split into hi + mid / 8 + lo / 64 of e5m2 numbers: hi and mid are cut after two fraction bits (toward zero; an
e5m2 number is the upper byte of an fp16 one), lo is rounded to the nearest. A row of Q, scaled to a largest element in [128, 256), is hi + lo / 32 of e4m3 numbers, both rounded to the
nearest."""

import numpy as np
import pytest

from oracle.paged_fp8 import TABLE, round_e4m3


def cut(x):
    """Toward zero to e5m2: fp16's upper byte."""
    return (x.astype(np.float16).view(np.uint16) & 0xFF00).view(np.float16).astype(np.float64)


def nearest_e5m2(x):
    """Two fraction bits, steps of 2^-16 at least; ties to even."""
    e = np.maximum(np.frexp(x)[1] - 1, -14)
    step = 2.0 ** (e - 2)
    return np.rint(x / step) * step


def split_p(p):
    h = p.astype(np.float16).astype(np.float64)
    hi = cut(h)
    r = (h - hi) * 8
    assert np.array_equal(r.astype(np.float16).astype(np.float64), r)  # (what the kernel computes in fp16 is exact)
    mid = cut(r)
    r = (r - mid) * 8
    assert np.array_equal(r.astype(np.float16).astype(np.float64), r)
    lo = nearest_e5m2(r)
    assert max(hi.max(), mid.max(), lo.max()) <= 57344  # e5m2's largest number
    return hi + mid / 8 + lo / 64


def every_p():
    """Every fp16 number from 0 to 2^15, the middles between two, and a step of fp32 beside each middle."""
    h = np.arange(0x7801, dtype=np.uint16).view(np.float16).astype(np.float64)
    mid = ((h[:-1] + h[1:]) / 2).astype(np.float32)
    beside = [np.nextafter(mid, np.float32(s)).astype(np.float64) for s in (0, 1e9)]
    return np.concatenate([h, mid.astype(np.float64), *beside])


def test_probabilities_keep_their_precision_far_below_the_largest():
    """Where the row's largest is 2^7 at least: 1.25 x 2^-23 of what is too small for the relative bound is 1.25 x 2^-30 of the largest."""
    p = every_p()
    binade = 2.0 ** (np.frexp(np.where(p == 0, 2.0**-60, p))[1] - 1)
    assert (np.abs(split_p(p) - p) <= np.maximum(1.25 * 2.0**-9 * binade, 1.25 * 2.0**-23)).all()
    one = np.abs(split_p(p) - p) / np.where(p == 0, 1, p)
    assert one[p >= 2.0**-13].max() <= 1.25 * 2.0**-9  # a key of 2^-20 of the largest


def test_the_largest_error_of_a_probability():
    """1.1 x 2^-9 of itself, which is more than lo's rounding alone (2^-9): down to 2^-13, which is 2^-20 of a row's largest."""
    p = every_p()
    p = p[p >= 2.0**-13]
    worst = (np.abs(split_p(p) - p) / p).max()
    assert 2.0**-9 < worst <= 1.1 * 2.0**-9


@pytest.mark.parametrize("top", [128.0, 191.0, 255.0])
def test_elements_of_q_are_exact_to_the_14th_binade_below_the_largest(top):
    """Every bf16 number up to the row's largest, binade by binade; the first that are off are off by 2^-22 of the largest at most."""
    nearest = lambda x: TABLE[round_e4m3(x)]  # noqa: E731
    for k in range(40):
        x = 2.0 ** (7 - k) * (1 + np.arange(128) / 128)
        x = x[x <= top]
        hi = nearest(x)
        off = np.abs(hi + nearest((x - hi) * 32) / 32 - x)
        assert (off.max() > 0) == (k > 14)
        assert off.max() <= 2.0**-22 * top
