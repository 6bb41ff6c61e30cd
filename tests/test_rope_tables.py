"""The rotary tables against 60-digit decimal arithmetic, at the positions where
their last bits count.  A frequency is computed in 64-bit significands: base,
factor and the other arguments are exact, and power, products, quotients and
the division by 2 pi round eight times at most, each 2^-64 of the value (the
power 2^-63); a clamped blend multiplies that by T f / 2 pi / (high - low), at
most 11 in these cases where its weight is not 0 or 1 (low 1, high 4 or 32: T
f / 2 pi below high, so high / (high - low), at most 4/3, plus one).  Together
below 2^-60 f / 2 pi, and the rounding to 2^-64ths."""

from decimal import Decimal, getcontext

import pytest

from bit_kv_cache_tq_b200 import tq

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803")


def _turns(r, base, kind, factor, low, high, trained, borders):
    """f_i / 2 pi of every pair, from the definition in include/tq.h."""
    base, factor, low, high, trained = map(Decimal, (base, factor, low, high, trained))
    b = base * factor ** (Decimal(r) / (r - 2)) if kind == tq.TQ_ROPE_SCALE_BASE and r > 2 else base
    out = []
    for i in range(r // 2):
        f = b ** (Decimal(-2 * i) / r)
        if kind == tq.TQ_ROPE_SCALE_LINEAR:
            f /= factor
        elif kind == tq.TQ_ROPE_SCALE_WAVELENGTH:
            s = min(Decimal(1), max(Decimal(0), (trained * f / (2 * PI) - low) / (high - low)))
            f = (1 - s) * f / factor + s * f
        elif kind == tq.TQ_ROPE_SCALE_RAMP:
            s = min(Decimal(1), max(Decimal(0), (i - borders[0]) / max(borders[1] - borders[0], Decimal("0.001"))))
            f = s * f / factor + (1 - s) * f
        out.append(f / (2 * PI))
    return out


def _borders(r, base, low, high, trained):
    def at(n):
        return r * (Decimal(trained) / (2 * PI * Decimal(n))).ln() / (2 * Decimal(base).ln())
    lo, hi = at(high).to_integral_value("ROUND_FLOOR"), at(low).to_integral_value("ROUND_CEILING")
    return max(Decimal(0), lo), min(Decimal(r - 1), hi)


@pytest.mark.parametrize("rotary", [2, 64, 90, 128, 256])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1.0e7])
@pytest.mark.parametrize("kind", ["NONE", "LINEAR", "BASE", "WAVELENGTH", "RAMP"])
def test_angles_at_the_farthest_positions(kind, base, rotary):
    """The table times a position, modulo one turn, is the angle to 2^-29 of a turn at both ends of int32 (the kernels
    round it to fp32, 2^-26 of a turn): 2^31 (2^-60 / 2 pi + 2^-65) is below 2^-31.6."""
    getcontext().prec = 60
    kind = getattr(tq, "TQ_ROPE_SCALE_" + kind)
    factor, low, high, trained = 8.0, 1.0, 32.0 if kind == tq.TQ_ROPE_SCALE_RAMP else 4.0, 8192.0
    rope = tq.tq_rope_init(rotary, tq.TQ_ROPE_HALF, base, kind, factor, low, high, trained)
    want = _turns(rotary, base, kind, factor, low, high, trained, _borders(rotary, base, low, high, trained))
    for i, w in enumerate(want):
        for position in (1, 2 ** 31 - 1, -2 ** 31):
            got = Decimal((rope.turns[i] * position) % 2 ** 64) / 2 ** 64
            off = (got - w * position) % 1
            assert min(off, 1 - off) <= Decimal(2) ** -29, (i, position)
        off = (Decimal(rope.turns[i]) / 2 ** 64 - w) % 1
        assert min(off, 1 - off) <= w * Decimal(2) ** -60 + Decimal(2) ** -65
