"""Rotary frequencies in 64-bit fixed-point turns: the nearest number, from radians in 64 bits."""
import math
from decimal import Decimal, getcontext

import pytest

from mla_decode_attention_03_gb300 import ops


def two_pi(digits):
    """2 pi to that many digits, by the arithmetic-geometric mean (Gauss, Legendre)."""
    getcontext().prec = digits + 10
    a, b, t, p = Decimal(1), 1 / Decimal(2).sqrt(), Decimal(1) / 4, Decimal(1)
    while abs(a - b) > Decimal(10) ** -(digits // 2 + 5):
        a, b, t, p = (a + b) / 2, (a * b).sqrt(), t - p * ((a - b) / 2) ** 2, 2 * p
    return (a + b) ** 2 / (2 * t)


@pytest.mark.parametrize("f", [1.0, 10000.0 ** (-2 / 64), 10000.0 ** (-62 / 64), math.pi / 2, 2 * math.pi, 1e-300, 5e-324, 1e6,
                               -0.5, 0.0, 1e22, 1.7e308, -1.7e308])
def test_turns_are_the_nearest(f):
    turn = two_pi(400)
    got = ops.Rotary(2, frequencies=[f], device="cpu").turns.item() % (1 << 64)
    off = (Decimal(f) / turn - Decimal(got) / Decimal(2) ** 64) % 1
    off = min(abs(off), abs(1 - abs(off)))
    assert off <= Decimal(2) ** -65 * (1 + Decimal(10) ** -9)


def test_turns_of_a_model():
    turn = two_pi(60)
    for kw in ({}, dict(factor=40.0, original_length=4096), dict(dim=128, base=500000.0)):
        rotary = ops.Rotary(device="cpu", **kw)
        for t, f in zip(rotary.turns.tolist(), rotary.frequencies):
            assert abs(Decimal(t % (1 << 64)) - Decimal(f) / turn * 2 ** 64) <= Decimal("0.5000001")
