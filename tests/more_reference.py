"""Plain 64-bit implementations of rotary positions, e2m1 groups and attention with formed scores
(include/bitdelta_step.h), on the host: test infrastructure, sharing no code with the kernels."""

import numpy as np

# the eight non-negative e2m1 values, by code
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def rotary(x, positions, frequencies, turned, interleaved, gain=1.0):
    """x [T, heads, dim] float64, frequencies in radians per position -> (turned rows, sum of magnitudes behind each)."""
    y, size = x.copy(), np.abs(x)
    t = positions.astype(np.float64)[:, None, None] * np.asarray(frequencies, np.float64)[None, None, :]
    cos, sin = np.cos(t) * gain, np.sin(t) * gain
    first = slice(0, turned, 2) if interleaved else slice(0, turned // 2)
    second = slice(1, turned, 2) if interleaved else slice(turned // 2, turned)
    a, b = x[..., first], x[..., second]
    y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
    size[..., first] = size[..., second] = (np.abs(a) + np.abs(b)) * abs(gain)
    return y, size


def scale_byte4(amax):
    """The byte of the smallest power of two 2^e, e >= -125, with amax <= 6 * 2^e."""
    e = -125
    while amax > 6.0 * 2.0 ** e:
        e += 1
    return e + 127


def quantise4(rows):
    """[..., dim] float64 -> (codes 0..15 uint8 [..., dim], scale bytes [..., dim / 32]); codes of a group that holds
    something not finite are 0."""
    flat = rows.reshape(-1, 32)
    codes, bytes_ = np.zeros(flat.shape, np.uint8), np.empty(flat.shape[0], np.uint8)
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    for i, r in enumerate(flat):
        if not np.isfinite(r).all():
            bytes_[i] = 255
            continue
        bytes_[i] = scale_byte4(np.abs(r).max())
        y = np.abs(r) / 2.0 ** (int(bytes_[i]) - 127)
        lo, hi = np.searchsorted(mid, y, side="left"), np.searchsorted(mid, y, side="right")
        code = np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi))
        codes[i] = code | np.signbit(r) * 8
    return codes.reshape(rows.shape), bytes_.reshape(rows.shape[:-1] + (rows.shape[-1] // 32,))


def decode4(codes, bytes_):
    """Codes 0..15 [..., dim] and scale bytes [..., dim / 32] -> float64."""
    b = np.repeat(np.asarray(bytes_, np.float64), 32, axis=-1)
    with np.errstate(over="ignore"):
        v = E2M1[codes & 7] * 2.0 ** (b - 127)
    v = np.where(b == 255, np.nan, v)
    return np.where(codes >= 8, -v, v)


def pack4(codes):
    return codes[..., 0::2] | codes[..., 1::2] << 4


def unpack4(packed):
    return np.stack((packed & 15, packed >> 4), -1).reshape(packed.shape[:-1] + (packed.shape[-1] * 2,))
