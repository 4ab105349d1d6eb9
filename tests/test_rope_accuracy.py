"""The rotation's angles: the table's entries against integer arithmetic."""
import math
from fractions import Fraction

import exact_tiled_attention_21_gb300 as fa

PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
FREQS = [1.0, 0.75, 10000.0 ** -0.5, 10000.0 ** (-126.0 / 128), 1e-9, 3.0, 7.5, 123456.789, 2.0 ** -40]


def test_table_is_the_quotient_in_double_precision():
    """turns = inv_freq / (2 pi) as a double has it (the division's half step, 2^-53, and 2 pi's own: 2^-52 of the
    quotient), rounded to 2^-65; negative frequencies turn the other way by exactly as much."""
    got = fa.fa_rope_table(FREQS)
    for t, x in zip(got, FREQS):
        exact = Fraction(x) / (2 * PI)
        off = Fraction(t, 1 << 64) - (exact - math.floor(exact))
        off = min(abs(off), 1 - abs(off))
        assert off <= exact / (1 << 52) + Fraction(1, 1 << 65), x
    back = fa.fa_rope_table([-x for x in FREQS])
    assert [(a + b) % (1 << 64) for a, b in zip(got, back)] == [0] * len(FREQS)
