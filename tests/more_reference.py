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
    fine = np.isfinite(flat).all(1)
    y = np.abs(np.where(fine[:, None], flat, 0.0))
    m, e = np.frexp(y.max(1))                       # a = m 2^e, m from 1/2: 6 2^(e - 3) is three quarters of 2^e
    e = np.maximum(np.where(m > 0, e - 3 + (m > 0.75), -125), -125)
    y = y / 2.0 ** e[:, None].astype(np.float64)
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    lo, hi = np.searchsorted(mid, y, side="left"), np.searchsorted(mid, y, side="right")
    codes = np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi)) | np.signbit(flat) * 8
    codes = np.where(fine[:, None], codes, 0).astype(np.uint8)
    bytes_ = np.where(fine, e + 127, 255).astype(np.uint8)
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


def scores(q, k, scale, cap=0.0, slopes=None, position=0):
    """Formed scores [Hq, n] of queries [Hq, D] and their heads' keys [Hq, n, D], and the largest sum of |q k| scale."""
    with np.errstate(all="ignore"):
        prod = q[:, None, :] * k
        s = prod.sum(2) * scale
        a = np.abs(prod * scale).sum(2)
        if cap:
            s = cap * np.tanh(s / cap)
        if slopes is not None:
            s = s - slopes[:, None] * np.abs(position - np.arange(k.shape[1]))[None, :]
    return s, a[np.isfinite(a)].max(initial=0.0)


def attend(q, k_rows, v_rows, scale, cap=0.0, slopes=None, first=0, last=None, position=None):
    """One query token: q [Hq, D], rows [n, H, D] (float64) -> (out [Hq, D], lse [Hq], largest sum of |q k| scale over
    the tokens seen); tokens outside [first, last) are as if they were not there."""
    hq, d = q.shape
    n, h, _ = k_rows.shape
    last = n if last is None else min(last, n)
    first = max(first, 0)
    position = n - 1 if position is None else position
    if first >= last:
        return np.zeros((hq, d)), np.full(hq, -np.inf), 0.0
    pick = np.arange(hq) // (hq // h)
    seen = slice(first, last)
    k = k_rows[seen][:, pick].transpose(1, 0, 2)
    v = v_rows[seen][:, pick].transpose(1, 0, 2)
    s, reach = scores(q, k, scale, cap, slopes, position - first)
    with np.errstate(all="ignore"):
        top = s.max(1, keepdims=True)
        p = np.exp(s - top)
        out = (p[:, None, :] @ v)[:, 0] / p.sum(1)[:, None] if np.isfinite(v).all() else \
            (p[:, :, None] * v).sum(1) / p.sum(1)[:, None]
        return out, top[:, 0] + np.log(p.sum(1)), reach


def score_error(dim, reach, cap=0.0, slope_reach=0.0):
    """How far a score is off at most: dim products and sums and a few more, the capping's 2^-19 of what it caps (tanh is
    off by 2^-21 where its argument is past a quarter, and by less of its result below), the distance's product and sum."""
    u = 2.0 ** -24
    return (dim + 8) * u * reach + (2.0 ** -19 * min(reach, cap) if cap else 0.0) + 3 * u * slope_reach


def attend_prompt(q, k_rows, v_rows, scale, first, last, position, cap=0.0, slopes=None):
    """New tokens of one sequence: q [n, Hq, D], rows [len, H, D] (float64), per token its range of keys and its position
    -> (out [n, Hq, D], lse [n, Hq], largest sum of |q k| scale, and the weights' mean of |v| and root mean square share of
    it: sum p |v| / sum p and sqrt(sum (p v)^2) / sum p, both [n, Hq, D])."""
    n, hq, d = q.shape
    out, lse = np.zeros(q.shape), np.full((n, hq), -np.inf)
    mean, share, reach = np.zeros(q.shape), np.zeros(q.shape), 0.0
    group = hq // k_rows.shape[1]
    for t in range(n):
        lo, hi = max(0, int(first[t])), min(len(k_rows), int(last[t]))
        if lo >= hi:
            continue
        for h in range(k_rows.shape[1]):
            at = slice(h * group, h * group + group)
            k, v = k_rows[lo:hi, h], v_rows[lo:hi, h]
            slope = None if slopes is None else slopes[at]
            s, a = scores(q[t, at], np.broadcast_to(k, (group, *k.shape)), scale, cap, slope, int(position[t]) - lo)
            reach = max(reach, a)
            with np.errstate(all="ignore"):
                top = s.max(1, keepdims=True)
                p = np.exp(s - top)
                total = p.sum(1, keepdims=True)
                lse[t, at] = (top + np.log(total))[:, 0]
                p = p / total
                if np.isfinite(v).all():
                    out[t, at], mean[t, at], share[t, at] = p @ v, p @ np.abs(v), np.sqrt(p ** 2 @ v ** 2)
                else:
                    pv = p[:, :, None] * v
                    out[t, at], fine = pv.sum(1), np.where(np.isfinite(pv), pv, 0.0)
                    mean[t, at], share[t, at] = np.abs(fine).sum(1), np.sqrt((fine ** 2).sum(1))
    return out, lse, reach, mean, share
