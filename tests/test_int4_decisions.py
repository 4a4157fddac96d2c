"""The 4-bit append's arithmetic (append.cu: int4_scale, int4_pack8), step by step on the host, for
every largest value and for every pair of a scale and a value: its scales and codes are those of
the exact quotients."""
from fractions import Fraction

import numpy as np

import oracle

POSITIVE = np.arange(1, 0x7C00, dtype=np.uint16).view(np.float16).astype(np.float64)


def _fp32(x: Fraction) -> Fraction:
    """x > 0 to the nearest binary32 value (normal range), ties to even."""
    e = x.numerator.bit_length() - x.denominator.bit_length()
    if Fraction(2) ** e > x:
        e -= 1
    ulp = Fraction(2) ** (e - 23)
    n, rest = divmod(x, ulp)
    if rest * 2 > ulp or (rest * 2 == ulp and n % 2):
        n += 1
    return n * ulp


def _scales():
    x = np.zeros((len(POSITIVE), 128), np.float16)
    x[:, 5] = POSITIVE
    return oracle.int4_group_scale(x)[:, 0]


def test_the_corrected_quotient_is_the_rounded_one():
    """a / 7 by the reciprocal and the exact remainder, for every fp16 a; the roundings to bfloat16
    and fp16 that follow are the oracle's."""
    seventh = _fp32(Fraction(1, 7))
    for a in POSITIVE:
        a = Fraction(float(a))
        q0 = _fp32(a * seventh)
        rest = a - 7 * q0                         # (exact in binary32: a fused multiply-add)
        assert rest == 0 or _fp32(abs(rest)) == abs(rest)
        q = _fp32(rest * seventh + q0)
        assert q == _fp32(a / 7)
    assert (_scales() <= 2720).all() and (_scales()[POSITIVE >= 7 * 2.0 ** -24] > 0).all()


def test_every_pair_of_a_scale_and_a_value_gets_the_exact_code():
    """With any reciprocal within 2^-23 of 1 / s, which is what rcp.approx promises."""
    scales = np.unique(_scales())
    scales = scales[scales > 0]
    assert len(scales) > 2500
    pairs = 0
    for s in scales:
        exact = np.rint(POSITIVE / s)
        off = 2 * np.abs(POSITIVE - exact * s)    # (fp16 values and products of 11 bits: exact)
        near = POSITIVE < 16 * s
        assert ((off < s) | ((off == s) & (exact % 2 == 0)))[near].all()
        code = np.minimum(exact, 7)
        r0 = np.float32(1 / s)
        for r in (np.nextafter(r0, np.float32(0)), r0, np.nextafter(r0, np.float32(np.inf))):
            r = float(r)
            if abs(r * s - 1) > 2.0 ** -23:
                continue
            y = POSITIVE * r                      # (35 bits: exact)
            # the usual way: to a multiple of 2^-13, then to a whole number
            sure = y.astype(np.float32) < np.float32(7.4)
            got = np.rint(np.rint(y[sure] * 8192) / 8192)
            assert (got <= 7).all() and np.array_equal(got, code[sure]), s
            # value by value, which any of a group may take
            ca = np.rint(np.minimum(y.astype(np.float32), np.float32(8))).astype(np.float64)
            up, down, odd = s * (ca + 0.5), s * (ca - 0.5), ca % 2 == 1
            mag = ca.copy()
            mag[(POSITIVE > up) | ((POSITIVE == up) & odd)] += 1
            less = (POSITIVE < down) | ((POSITIVE == down) & odd)
            mag[less] = ca[less] - 1
            assert np.array_equal(np.minimum(mag, 7), code), s
            pairs += len(POSITIVE)
    assert pairs > 10 ** 8
