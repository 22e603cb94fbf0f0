"""How exact the angles of rotary positions are, at any position."""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import tenant_serving_amd as bd

DEV = "cuda:0"
U = 2.0 ** -24


def turn():
    """2 pi to 60 digits and more, by Machin's formula in whole numbers."""
    one = 10 ** 80

    def arctan(n):
        total = term = one // n
        k = 1
        while term:
            term //= -n * n
            k += 2
            total += term // k
        return total
    return Fraction(2 * 4 * (4 * arctan(5) - arctan(239)), one)


def test_steps_are_rounded_once():
    """Each is its frequency's part of a turn to half of 2^-64, so the farthest position's angle is off by 2^-34 of one."""
    assert abs(turn() - Fraction(2 * math.pi)) < Fraction(1, 2 ** 50)
    for kw in (dict(), dict(scaling="linear", factor=3.0), dict(frequencies=[1.0, 0.7, 1e-9, 123456.789, -0.25, 2.0 ** 20, 3.0, 0.0])):
        a = bd.bd_rotary_angles(16, 500000.0, device="cpu", **kw)
        for s, f in zip(a.steps.tolist(), a.frequencies):
            off = (s - Fraction(f) / turn() * 2 ** 64) % 2 ** 64
            assert min(off, 2 ** 64 - off) <= Fraction(51, 100), f
