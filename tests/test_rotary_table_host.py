"""Tables of rotations against exact arithmetic (60 decimal digits, no GPU): every entry is the nearest
64-bit fraction of a turn, so that angles are as exact at the last position of int32 as at the first."""
import ctypes
import math
from decimal import Decimal, getcontext

import pytest

import exact_io_aware_16_gb300 as fa
from exact_io_aware_16_gb300 import build as fabuild

PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


@pytest.fixture(scope="module")
def lib():
    getcontext().prec = 60
    fabuild.build()
    return fa.library()


def exact(rot, base, scaling, factor, original, low, high):
    """Turns a position times 2^64 of each pair."""
    B, F, out = Decimal(base), Decimal(factor), []
    at = lambda t: rot * math.log(original / (2 * math.pi * t)) / (2 * math.log(base))  # noqa: E731
    if scaling == 4:
        first, last = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
    for i in range(rot // 2):
        f = B ** (Decimal(-2 * i) / rot)
        if scaling == 1:
            f /= F
        elif scaling == 2:
            f *= F ** (Decimal(-2 * i) / (rot - 2))
        elif scaling >= 3:
            if scaling == 3:
                g = (Decimal(original) * f / (2 * PI) - Decimal(low)) / (Decimal(high) - Decimal(low))
            else:
                g = 1 - Decimal(i - first) / max(Decimal(last - first), Decimal(1e-3))
            g = min(max(g, Decimal(0)), Decimal(1))
            f = g * f + (1 - g) * f / F
        out.append(f / (2 * PI) * 2 ** 64)
    return out


@pytest.mark.parametrize("base", (10000.0, 500000.0, 1.5, 1e7 / 3, 1e30))
@pytest.mark.parametrize("scaling,factor", [(0, 1.0), (1, 8.0), (1, 1.7), (2, 4.0), (2, 3.3), (3, 8.0), (3, 1.1), (4, 16.0), (4, 5.3)])
@pytest.mark.parametrize("rot", (16, 48, 64, 128))
def test_entries_are_the_nearest(lib, rot, scaling, factor, base):
    args = (rot, base, scaling, factor, 4096.0, 1.0, 32.0)
    table = (ctypes.c_ulonglong * (rot // 2))()
    assert lib.fa_rotary_table(table, *args) == 0
    for got, want in zip(table, exact(*args)):
        # half a unit, and 2^-100 of the value for the arithmetic of two doubles
        assert abs(Decimal(got) - want) <= Decimal("0.5") + want * Decimal(2) ** -90


def test_angles_at_the_last_position(lib):
    """2^31 times half a unit is 2^-34 of a turn."""
    table = (ctypes.c_ulonglong * 64)()
    assert lib.fa_rotary_table(table, 128, 10000.0, 0, 1.0, 0.0, 1.0, 32.0) == 0
    for i, t in enumerate(table):
        want = Decimal(10000) ** (Decimal(-2 * i) / 128) / (2 * PI) * (2 ** 31 - 1)
        got = Decimal((t * (2 ** 31 - 1)) % 2 ** 64) / 2 ** 64
        off = (got - want) % 1
        assert min(abs(off), abs(1 - abs(off))) <= Decimal(2) ** -33
