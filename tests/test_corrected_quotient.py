"""The quotient by product, residual and correction that the 8-bit kernels form in
place of a division gives the division's E4M3 codes: exact arithmetic over every
pair that could differ.

r = fp32(1 / s), z0 = fp32(x r), t = fp32(x - z0 s), z = fp32(z0 + t r).  With
relative errors |e| <= 2^-24 of r, z0 and t, z before its rounding is x / s times
1 - (e1 + e2 + e1 e2)(e1 + e3 + e1 e3), so it is off by at most 2^-46 (1 + 2^-22).
z and fp32(x / s) then differ only if x / s is that close to the middle B of two
neighbouring fp32 numbers, and their codes only if one of these is a border M of
E4M3's rounding (at most 5 significant bits).  In units where x and s are 24-bit
integers and B a 25-bit one, N = M 2^20 +- 1, that is |x 2^j - s N| <= 8: the low 20
bits of s are within 8 of 0.  All of these s (and a margin), all borders and the x
nearest to s B are gone through."""

from fractions import Fraction as F


def rn24(v):
    """Nearest number of 24 significant bits, ties to even."""
    if v == 0:
        return F(0)
    a = abs(v)
    e = a.numerator.bit_length() - a.denominator.bit_length()
    if F(2) ** e > a:
        e -= 1
    u = F(2) ** (e - 23)
    n, rest = divmod(a / u, 1)
    n = int(n) + (rest > F(1, 2) or (rest == F(1, 2) and int(n) % 2 == 1))
    return n * u if v > 0 else -n * u


def test_same_side_of_every_border_as_the_division():
    pairs = 0
    for s in (c * 2 ** 20 + e for c in range(8, 17) for e in range(-10, 11)):
        if not 2 ** 23 <= s < 2 ** 24:
            continue
        r = rn24(F(1, s))
        for m5 in range(16, 32):
            for side in (1, -1):
                step = F(1, 2 ** (20 if m5 == 16 and side < 0 else 19))   # fp32 step on that side of m5
                scale = F(1)
                while s * (m5 + side * step / 2) * scale >= 2 ** 24:
                    scale /= 2
                border = m5 * scale
                x0 = round(s * (m5 + side * step / 2) * scale)
                for x in range(x0 - 2, x0 + 3):
                    if not 2 ** 23 <= x < 2 ** 24:
                        continue
                    z0 = rn24(x * r)
                    z, q = rn24(z0 + rn24(x - z0 * s) * r), rn24(F(x, s))
                    assert (z > border) - (z < border) == (q > border) - (q < border), (s, x, m5)
                    pairs += 1
    assert pairs > 20000


def test_quotients_of_16_bit_values_with_reciprocals_up_to_two_units_off():
    """The few-token layer's input: bf16 values x over s = fp32(amax / 448), with a
    reciprocal r within two fp32 steps of 1 / s (a hardware reciprocal of one step
    and a Newton step).  The quotient by product, residual and correction is the IEEE
    quotient for every mantissa of x and of amax.  (Powers of two scale every step
    exactly where the code is not 0: x > 2^-11 s, s >= 2^-90, so the residual's last
    bit is at 2^-149 or above.)"""
    for ma in range(128, 256):
        s = rn24(F(ma, 448))
        r0 = rn24(1 / s)
        ulp = F(1, 2 ** 23)
        while r0 < ulp * 2 ** 23:
            ulp /= 2
        quotients = [(mx, rn24(mx / s)) for mx in range(128, 256)]
        for r in (r0 + d * ulp for d in range(-2, 3)):
            for mx, q in quotients:
                z0 = rn24(mx * r)
                assert rn24(z0 + rn24(mx - z0 * s) * r) == q, (ma, mx)


def test_tile_scale_without_division():
    """amax / 448 from the rounded reciprocal and one residual correction is the IEEE
    quotient for every mantissa of amax (the residual is exact and clear of underflow
    for amax >= 2^-110)."""
    import numpy as np
    a = np.arange(2 ** 23, 2 ** 24, dtype=np.float64)
    r = float(np.float32(1) / np.float32(448))
    f32 = lambda v: v.astype(np.float32).astype(np.float64)   # noqa: E731
    q = f32(a * r)                        # 48-bit products: exact before the rounding
    res = f32(a - q * 448.0)              # both exact, and so is their difference
    p = res * r                           # at most 24 + 24 bits: exact
    total = q + p
    # the sum's own rounding to 53 bits must not decide the rounding to 24
    lost = (q - total) + p
    low = total.view(np.uint64) & np.uint64(2 ** 29 - 1)
    assert not np.any((lost != 0) & (low == 2 ** 28))
    assert np.array_equal(total.astype(np.float32), a.astype(np.float32) / np.float32(448))
