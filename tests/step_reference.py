"""Plain 64-bit implementations of the operators between the linears of a step (include/bitdelta_step.h), on the
host: test infrastructure, sharing no code with the kernels.  e4m3 rounding goes through the table of the format's
values, scales through exact halving and doubling."""

import numpy as np
import torch

# the 127 non-negative finite e4m3 values, by code
E4M3 = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)])
assert E4M3[-1] == 448.0


def bf16(x64):
    """float64 -> nearest bf16, by way of fp32 (a test's inputs keep clear of double rounding or are fp32 already)."""
    return torch.from_numpy(np.ascontiguousarray(x64)).float().to(torch.bfloat16)


def scale_byte(amax):
    """The byte of the smallest power of two 2^e, e >= -111, with amax <= 448 * 2^e."""
    e = -111
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return e + 127


def encode(x, byte):
    """Codes of the values x (float64) at a scale byte: nearest, ties to the even code, NaN code for what is not
    finite."""
    y = np.abs(x) / 2.0 ** (int(byte) - 127)
    mid = (E4M3[1:] + E4M3[:-1]) / 2
    fine = np.isfinite(x)
    y = np.where(fine, y, 0.0)
    lo = np.searchsorted(mid, y, side="left")    # a value on a midpoint: the code below it
    hi = np.searchsorted(mid, y, side="right")   # the code above it
    code = np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi))
    code = np.where(fine, code, 127)
    return (code | (np.signbit(x) & fine) * 128).astype(np.uint8)


def decode(codes, byte):
    c = codes.astype(np.int64)
    v = np.where((c & 127) == 127, np.nan, np.append(E4M3, np.nan)[c & 127])
    return np.where(c >= 128, -v, v) * 2.0 ** (np.asarray(byte, np.float64) - 127)


def quantise(rows):
    """[..., n] float64 -> (codes uint8, scale bytes [...]), one group per row."""
    flat = rows.reshape(-1, rows.shape[-1])
    codes, bytes_ = np.empty(flat.shape, np.uint8), np.empty(flat.shape[0], np.uint8)
    for i, r in enumerate(flat):
        fine = np.abs(r[np.isfinite(r)])
        bytes_[i] = scale_byte(fine.max() if fine.size else 0.0)
        codes[i] = encode(r, bytes_[i])
    return codes.reshape(rows.shape), bytes_.reshape(rows.shape[:-1])


def to64(t):
    return t.detach().cpu().double().numpy()


def rms_norm(x, gain, eps, residual=None, ids=None):
    """(y float64, residual_out in its type).  x, gain, residual: torch tensors [M, d], [V, d]."""
    h = x.detach().cpu().float()
    res_out = None
    if residual is not None:
        res_out = (h + residual.detach().cpu().float()).to(residual.dtype)  # the fp32 sum, rounded to the type
        h = res_out
    h = to64(h)
    gain = to64(gain)
    ids = np.zeros(h.shape[0], int) if ids is None else ids.cpu().numpy()
    with np.errstate(all="ignore"):
        y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    known = (ids >= 0) & (ids < gain.shape[0])
    y = y * gain[np.where(known, ids, 0)]
    y[~known] = np.nan
    return y, res_out


def attend(q, k_rows, v_rows, scale):
    """One sequence: q [Hq, D], rows [n, H, D] (float64) -> (out [Hq, D], lse [Hq], largest sum of |q k| scale)."""
    hq, d = q.shape
    n, h, _ = k_rows.shape
    out, lse, reach = np.zeros((hq, d)), np.full(hq, -np.inf), 0.0
    if n == 0:
        return out, lse, reach
    group = hq // h
    for i in range(hq):
        k, v = k_rows[:, i // group], v_rows[:, i // group]
        with np.errstate(all="ignore"):
            s = (k * q[i]).sum(1) * scale
            top = s.max()
            p = np.exp(s - top)
            out[i] = (p[:, None] * v).sum(0) / p.sum()
            lse[i] = top + np.log(p.sum())
            a = np.abs(k * q[i] * scale).sum(1)
        reach = max(reach, a[np.isfinite(a)].max(initial=0.0))
    return out, lse, reach
