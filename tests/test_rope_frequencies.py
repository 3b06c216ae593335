"""Frequencies of the ramp scaling against values worked out apart from the code."""
from decimal import Decimal, getcontext

import exact_attention_17_gb300 as fa2

getcontext().prec = 60
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494")


def expected(r, base, factor, length, fast, slow):
    """Pair i turns length f_i / (2 pi) times within the length.  The first pair that turns at most `fast`
    times, before rounding, is where r ln(length / (2 pi fast)) / (2 ln base) lies: the ramp starts at the
    whole number below and ends at the one above the same for `slow`."""
    base, factor, length = Decimal(base), Decimal(factor), Decimal(length)

    def at(turns):
        return r * (length / (2 * PI * Decimal(turns))).ln() / (2 * base.ln())

    low = max(int(at(fast).to_integral_value("ROUND_FLOOR")), 0)
    high = min(int(at(slow).to_integral_value("ROUND_CEILING")), r - 1)
    out = []
    for i in range(r // 2):
        f = (-(Decimal(2 * i) / r) * base.ln()).exp()
        share = min(Decimal(1), max(Decimal(0), Decimal(i - low) / max(high - low, Decimal("0.001"))))
        out.append(f * ((1 - share) + share / factor))
    return low, high, out


def test_ramp():
    # r = 128, base 10000, length 4096, turns 32 and 1: 128 ln(4096 / 201.06) / (2 ln 10000) = 20.95 and
    # 128 ln(4096 / 6.2832) / 18.4207 = 45.03, so the pairs 20 .. 46
    low, high, want = expected(128, 10000, 4, 4096, 32, 1)
    assert (low, high) == (20, 46)
    # half way, pair 33: 10000^(-66/128) (1 - 13/26 + 13/26/4) = 0.0086596... * 0.625
    assert abs(want[33] - Decimal(10000) ** (Decimal(-66) / 128) * Decimal("0.625")) < Decimal("1e-30")
    for args in ((128, 10000, 4, 4096, 32, 1), (64, 10000, 8, 4096, 32, 1), (64, 500000, 8, 8192, 4, 1),
                 (48, 1000000, 40, 32768, 32, 1), (16, 10000, 2, 100, 32, 1), (8, 100, 4, 4096, 32, 1)):
        r, base, factor, length, fast, slow = args
        got = fa2.rope_inv_freq(r, base=base, scaling="ramp", factor=factor, original_length=length, beta_fast=fast,
                                beta_slow=slow).tolist()
        low, high, want = expected(*args)
        assert any(f * factor > w * Decimal("1.0001") and w < f * Decimal("0.9999")
                   for f, w in zip([Decimal(base) ** (Decimal(-2 * i) / r) for i in range(r // 2)], want)), args
        for i, (a, b) in enumerate(zip(got, want)):
            # in half steps of 2^-53: the power 2, its exponent's rounding times the exponent times ln(base) 14, the
            # share's rounding at most factor - 1 of the sum, and five more operations
            assert abs(Decimal(a) - b) <= b * (20 + factor) * Decimal(2) ** -53, (args, i)
