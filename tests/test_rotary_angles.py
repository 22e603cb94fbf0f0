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


@pytest.mark.gpu
@pytest.mark.parametrize("interleaved", [False, True])
def test_sine_and_cosine_at_any_position(interleaved):
    """Rows of (1, 0) turn into (cos t, sin t).  The phase is kept to 2^-32 of a turn (1.5e-9), what is left of the nearest
    quarter is rounded to fp32 as it is, by its factor and by their product: at most 3 u of pi / 4, 1.42e-7 with it.  The
    series end 2^-28 short and are rounded twice."""
    a = bd.bd_rotary_angles(64, 500000.0, interleaved=interleaved, device=DEV)
    gen = torch.Generator().manual_seed(2)
    pos = torch.cat([torch.arange(-3000, 3000), torch.randint(-2 ** 31, 2 ** 31, (20000,), generator=gen),
                     torch.tensor([2 ** 31 - 1, -2 ** 31])]).to(torch.int32)
    x = torch.zeros((len(pos), 1, 64), device=DEV)
    first = slice(0, None, 2) if interleaved else slice(0, 32)
    second = slice(1, None, 2) if interleaved else slice(32, None)
    x[..., first] = 1
    y = bd.bd_rotary(a, x, pos.to(DEV), dtype=torch.float32)[:, 0].cpu().double().numpy()
    # the phase in whole numbers, as a signed fraction of 2^64 of a turn
    with np.errstate(over="ignore"):
        phase = (pos.numpy().astype(np.int64)[:, None] * a.steps.cpu().numpy()[None, :]).astype(np.float64)
    t = phase * (2.0 * math.pi / 2.0 ** 64)     # off by 2^-52 of at most pi
    off = np.maximum(np.abs(y[:, first] - np.cos(t)), np.abs(y[:, second] - np.sin(t)))
    assert off.max() <= 1.42e-7 * math.sqrt(0.5) + 2.0 ** -28 + 2 * U, off.max()
