"""Python binding of rotary positions (include/bitdelta_step.h): the angles of a model's heads, made once, and the call
that turns a step's queries and keys by them, between the q and k linears and the cache.

Argument marshalling only; the turning runs in the library's HIP kernel, and there is no fallback.
"""

from __future__ import annotations

import ctypes
import math
from fractions import Fraction

import torch

from . import step
from .bitdelta import _check
from .step import _IN, _Pair, _any_on_rows, _index, _overlap, _plain, _rows, _same_gpu, _span, _tensor, _typed

_TURN = Fraction("6.283185307179586476925286766559005768394338798750211641949889")  # 2 pi


class bd_rotary_angles:
    """The angles of rotary positions: per pair of columns the part of a turn that a position adds, as a whole fraction
    of 2^64 turns on the device.

    The first `turned` columns of a head are turned in pairs (i, i + turned/2), or (2i, 2i+1) where interleaved.  Pair i
    has base^(-2i/turned) radians per position, for contexts longer than the trained one scaled by a method:

      "none"    not at all
      "linear"  all of them divided by factor
      "base"    base times factor^(turned/(turned-2)), which leaves the fastest pair and divides the slowest by factor
      "bands"   by how often a pair comes round within the trained context: up to `low` times divided by factor, from
                `high` times on left, between the two mixed in proportion

    or frequencies gives them (radians per position, [turned/2] numbers or a host float64 tensor).  gain multiplies what
    is turned."""

    def __init__(self, turned: int, base: float = 10000.0, *, interleaved: bool = False, scaling: str = "none",
                 factor: float = 1.0, trained: int | None = None, low: float = 1.0, high: float = 4.0,
                 gain: float = 1.0, frequencies=None, device="cuda"):
        if turned % 2 or not 2 <= turned <= 256:
            raise ValueError("turned must be even, 2..256 (got %r)" % turned)
        if not math.isfinite(gain):
            raise ValueError("gain must be finite (got %r)" % gain)
        if frequencies is None:
            frequencies = self._scaled(turned, base, scaling, factor, trained, low, high)
        else:
            frequencies = [float(x) for x in (frequencies.tolist() if isinstance(frequencies, torch.Tensor) else frequencies)]
        if len(frequencies) != turned // 2 or not all(abs(x) <= 2.0 ** 20 for x in frequencies):
            raise ValueError("frequencies must be %d numbers of at most 2^20 (got %s)" % (turned // 2, frequencies))
        # the low 64 bits, as the signed number that int64 holds; a float64's quotient would be off by 2^-56 of a turn,
        # which the farthest position makes 2^-25
        steps = [round(Fraction(x) / _TURN * 2 ** 64) & (1 << 64) - 1 for x in frequencies]
        self.steps = torch.tensor([x - (x >> 63 << 64) for x in steps], dtype=torch.int64, device=device)
        self.turned, self.interleaved, self.gain = turned, bool(interleaved), float(gain)
        self.frequencies = frequencies

    @staticmethod
    def _scaled(turned, base, scaling, factor, trained, low, high):
        if not (base > 0.0 and math.isfinite(base) and factor > 0.0 and math.isfinite(factor)):
            raise ValueError("base and factor must be above 0 (got %r, %r)" % (base, factor))
        if scaling == "base":
            if turned < 4:
                raise ValueError("scaling the base takes at least two pairs")
            base = base * factor ** (turned / (turned - 2))
        f = [base ** (-2.0 * i / turned) for i in range(turned // 2)]
        if scaling == "linear":
            return [x / factor for x in f]
        if scaling == "bands":
            if not trained or trained < 1 or not low < high:
                raise ValueError("bands need the trained context and low < high")
            keep = [min(1.0, max(0.0, (trained * x / (2.0 * math.pi) - low) / (high - low))) for x in f]
            return [x * s + x / factor * (1.0 - s) for x, s in zip(f, keep)]
        if scaling not in ("none", "base"):
            raise ValueError('scaling must be "none", "linear", "base" or "bands" (got %r)' % (scaling,))
        return f


class _RotaryRows(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("x_strides", _Pair), ("out_strides", _Pair),
                ("heads", ctypes.c_int32)]


_Table = _RotaryRows * 2


def _row_starts(t):
    """(address, [(step, n)] falling, bytes of a row) of a [n, heads, dim] tensor's rows, as _on_rows takes them; None
    where the steps do not each pass the smaller ones' extent."""
    size = t.element_size()
    row = extent = t.shape[2] * size
    steps = sorted((s * size, n) for s, n in zip(t.stride()[:2], t.shape[:2]) if n > 1)
    for s, n in steps:
        if s < extent:
            return None
        extent += s * (n - 1)
    return t.data_ptr(), steps[::-1], row


def _rows_apart(a, b):
    """Whether no row of a [n, heads, dim] tensor meets one of another."""
    if not _overlap(a, b):
        return True
    # views side by side in one buffer: tokens one step apart in both, each token's rows within a part of the step
    if a.shape[0] == b.shape[0] and a.stride(0) * a.element_size() == b.stride(0) * b.element_size() and a.shape[0] > 1:
        step = a.stride(0) * a.element_size()
        (a0, a1), (b0, b1) = _span(a[0]), _span(b[0])
        at = (b0 - a0) % step
        if a1 - a0 <= at and at + (b1 - b0) <= step:
            return True
    rows = _row_starts(a)
    if rows is None:
        return False
    starts = torch.tensor(b.data_ptr(), dtype=torch.int64)
    for n, s in zip(b.shape[:2], b.stride()):
        starts = starts[..., None] + torch.arange(n) * (s * b.element_size())
    return not _any_on_rows(*rows, starts, b.shape[2] * b.element_size())


def _same_rows(a, b):
    return a.data_ptr() == b.data_ptr() and a.dtype == b.dtype and a.shape == b.shape and a.stride() == b.stride()


def _refuse_rotary(angles, q, k, q_out, k_out, positions):
    """The checks of a rotary call's tensors that the ordinary one does without; raises or returns."""
    _plain("positions", positions, torch.int32, (q.shape[0],))
    named = [("q", q), ("k", k), ("q_out", q_out), ("k_out", k_out), ("positions", positions),
             ("the angles", angles.steps)]
    named = [(name, t) for name, t in named if t is not None]
    own = {"q_out": "q", "k_out": "k"}  # an output may be its own input
    for name, o in named:
        if name not in own or not o.numel():
            continue
        if _row_starts(o) is None:
            raise ValueError("rows of %s overlap (strides %s)" % (name, tuple(o.stride())))
        for other, x in named:
            if other == name or (other == own[name] and _same_rows(o, x)):
                continue
            if not _rows_apart(o, x if x.dim() == 3 else x.view(1, 1, -1)):
                raise ValueError("%s overlaps %s" % (name, other))
    _same_gpu(q.device, named)


def bd_rotary(angles: bd_rotary_angles, q: torch.Tensor, positions: torch.Tensor, k: torch.Tensor | None = None,
              q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
              dtype: torch.dtype = torch.bfloat16):
    """The rows of q [T, num_q_heads, head_dim], and of k [T, num_heads, head_dim] in the same launch, turned by their
    tokens' positions (int32 [T], any); (q', k'), or q' without k.

    q and k are bf16 or fp32 alike, with any token and head strides, head_dim a multiple of 16 up to 256.  The columns
    behind angles.turned stay.  q_out and k_out, where given, take the results in their one dtype, with any strides;
    q_out may be q itself and k_out k (turned in place), otherwise they lie apart from all else.  What is not given is
    allocated, in the other's dtype or `dtype`: bf16, as the cache and the attention take it, or fp32."""
    if not isinstance(angles, bd_rotary_angles):
        raise TypeError("angles must be a bd_rotary_angles")
    _tensor("q", q)
    if q.dim() != 3 or q.shape[2] % 16 or not 16 <= q.shape[2] <= 256:
        raise ValueError("q must be [n, num_q_heads, head_dim], head_dim a multiple of 16, 16..256 (got %s)"
                         % (tuple(q.shape),))
    dim, dev = q.shape[2], q.get_device()
    if dim < angles.turned:
        raise ValueError("the angles turn %d columns, heads have %d" % (angles.turned, dim))
    kind, qs, n, heads, _ = _rows("q", q, None, dim)
    pairs = [("q_out", q, q_out, qs, heads)]
    if k is not None:
        k_kind, ks, k_n, k_heads, _ = _rows("k", k, None, dim)
        if k_kind != kind or k_n != n:
            raise ValueError("q and k must have one dtype and one number of tokens")
        pairs.append(("k_out", k, k_out, ks, k_heads))
    elif k_out is not None:
        raise ValueError("k_out needs k")
    for given in (q_out, k_out):
        if given is not None:
            _tensor("q_out and k_out", given)
            dtype = given.dtype
            break
    out_kind = _IN.get(dtype)
    if out_kind is None:
        raise TypeError("results are torch.bfloat16 or torch.float32 (got %s)" % (dtype,))
    strides = []
    for name, x, o, _, count in pairs:
        if not 1 <= count <= 65535:
            raise ValueError("need 1..65535 heads (got %d)" % count)
        if o is None:
            strides.append(_Pair(count * dim, dim))
        elif _typed(name, o, _IN) != out_kind or o.shape != x.shape:
            raise ValueError("%s must be %s of shape %s (got %s %s)" % (name, dtype, tuple(x.shape), o.dtype, tuple(o.shape)))
        else:
            strides.append(_rows(name, o, count, dim)[1])
    if not (_index("positions", positions, n, dev) and dev >= 0 and (k is None or k.get_device() == dev)
            and angles.steps.get_device() == dev and q_out is None and k_out is None):
        _refuse_rotary(angles, q, k, q_out, k_out, positions)
    if step._current_device() != dev:
        with torch.cuda.device(dev):
            return bd_rotary(angles, q, positions, k, q_out, k_out, dtype)
    lib = step._declared or step._library()
    table, outs = _Table(), []
    for i, (_, x, o, xs, count) in enumerate(pairs):
        if o is None:
            o = torch.empty(x.shape, dtype=dtype, device=x.device)
        outs.append(o)
        table[i] = _RotaryRows(x.data_ptr(), o.data_ptr(), xs, strides[i], count)
    st = lib.bd_rotary(table, len(pairs), kind, out_kind, dim, angles.turned, angles.interleaved, positions.data_ptr(),
                       angles.steps.data_ptr(), angles.gain, n, step._stream_of(dev))
    if st:
        _check(lib, "bd_rotary", st)
    return tuple(outs) if k is not None else outs[0]
