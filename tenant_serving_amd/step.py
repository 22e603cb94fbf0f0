"""Python binding of the operators between the linears of a step
(include/bitdelta_step.h), same names.

Argument marshalling only: shape, dtype, stride and device checks, output and
workspace allocation with torch, and the current HIP stream of the tensors'
device.  Every step of the computation runs in the library's HIP kernels;
there is no fallback.

A step of a served model runs, per layer: ``bd_rms_norm`` (the residual added,
each token normed with its variant's gain), the q, k, v linears, ``bd_rotary``
where the model has rotary positions, ``bd_kv_write``, ``bd_attend``, the
output linear, ``bd_rms_norm`` again and the remaining linears.
"""

from __future__ import annotations

import ctypes
import functools
import math
from bisect import bisect_right

import torch

from .bitdelta import _check, _workspace, library

BD_BF16, BD_FP32, BD_E4M3, BD_E2M1 = 0, 1, 2, 4
_IN = {torch.bfloat16: BD_BF16, torch.float32: BD_FP32}
_INT = torch.int32
_HELD = {torch.bfloat16: BD_BF16, torch.float8_e4m3fn: BD_E4M3, torch.float4_e2m1fn_x2: BD_E2M1}
_declared = None
# the current stream's handle and device as plain numbers: a call of a few microseconds on the GPU has no room for the
# objects around them (torch.cuda.current_stream takes 1.9 us, this 0.1)
_stream_of = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
              or (lambda index: torch.cuda.current_stream(index).cuda_stream))
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


class _KV(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("type", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64)]


class _Scores(ctypes.Structure):
    _fields_ = [("cap", ctypes.c_float), ("slopes", ctypes.c_void_p), ("first", ctypes.c_void_p),
                ("last", ctypes.c_void_p)]


_Pair = ctypes.c_int64 * 2
_NO_END = 1 << 64
_SIZE = (2, 4, 1)  # bytes of a value, by its type


def declare(lib):
    p, i32, i64, f, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.bd_rms_norm.argtypes = [p, i32, p, p, i32, p, i32, i32, p, f, p, i32, p, i64, i64, p]
    lib.bd_kv_write.argtypes = [p, p, p, p, p, i32, p, i64, p]
    lib.bd_kv_read.argtypes = [p, p, i64, p, p, p]
    lib.bd_attend.argtypes = [p, p, i32, p, i32, p, i64, i64, p, i64, f, p, p, p, sz, p]
    lib.bd_attend_scores.argtypes = [p, p, i32, p, i32, p, i64, i64, p, i64, f, p, p, p, p, sz, p]
    lib.bd_attend_prompt.argtypes = [p, p, p, i32, i64, p, i64, i64, p, p, i64, f, p, p, p, p, sz, p]
    lib.bd_rotary.argtypes = [p, i32, i32, i32, i32, i32, i32, p, p, f, i64, p]
    for n in ("rms_norm", "rotary", "kv_write", "kv_read", "attend", "attend_scores", "attend_prompt"):
        getattr(lib, "bd_" + n).restype = ctypes.c_int
    lib.bd_attend_workspace_bytes.argtypes = [i64] * 6
    lib.bd_attend_workspace_bytes.restype = sz
    lib.bd_attend_prompt_workspace_bytes.argtypes = [i64] * 7
    lib.bd_attend_prompt_workspace_bytes.restype = sz
    return lib


def _library():
    global _declared
    if _declared is None:
        _declared = declare(library())
    return _declared


def _tensor(name, t):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)


def _typed(name, t, types):
    _tensor(name, t)
    got = types.get(t.dtype)
    if got is None:
        raise TypeError("%s must be one of %s (got %s)" % (name, ", ".join(str(d) for d in types), t.dtype))
    return got


def _plain(name, t, dtype, shape):
    """A contiguous tensor of this dtype and shape."""
    _tensor(name, t)
    if t.dtype != dtype:
        raise TypeError("%s must be %s (got %s)" % (name, dtype, t.dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have shape %s (got %s)" % (name, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _same_gpu(device, named):
    if device.type != "cuda":
        raise ValueError("tensors must be on a GPU (got %s); there is no CPU path" % device)
    for name, t in named:
        if t is not None and t.device != device:
            raise ValueError("%s is on %s, expected %s" % (name, t.device, device))


def _span(t):
    """The addresses that a tensor reaches, gaps of its strides included."""
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size()


def _overlap(a, b):
    (a0, a1), (b0, b1) = _span(a), _span(b)
    return a0 < b1 and b0 < a1


def _at(t):
    return t.data_ptr() if t is not None else None


def _on_rows(base, steps, row, lo, hi):
    """Whether the addresses [lo, hi) meet rows of `row` bytes that start at base plus any number i < n of each step
    (step, n) of steps, which fall, each past the extent of all smaller ones."""
    left = hi - 1 - base
    if left < 0 or lo >= hi:
        return False
    last = base   # where the last row that starts before hi does
    for step, n in steps:
        i = min(n - 1, left // step)
        last += i * step
        left -= i * step
    return last + row > lo


def _any_on_rows(base, steps, row, starts, size):
    """_on_rows of any [start, start + size) of an int64 tensor of starts."""
    left = starts + (size - 1 - base)
    reach = left >= 0
    last = torch.full_like(starts, base)
    for step, n in steps:
        i = torch.div(left, step, rounding_mode="floor").clamp_(0, n - 1)
        last += i * step
        left -= i * step
    return bool((reach & (last + row > starts)).any())


def _apart(kv, lo, hi):
    """Whether the addresses [lo, hi) are outside all spans of the cache's arrays."""
    i = bisect_right(kv._bounds, lo)
    return not i & 1 and (i == len(kv._bounds) or hi <= kv._bounds[i])


def _refuse_on_cache(kv, named):
    """Raises where a tensor's rows (its last axis is contiguous) meet what the cache holds; the gaps of the cache's
    strides, and of the tensor's own, are not held."""
    for name, t in named:
        if not t.numel() or _apart(kv, *_span(t)):
            continue
        size = t.element_size()
        starts = torch.tensor(t.data_ptr(), dtype=torch.int64)
        for n, s in zip(t.shape[:-1], t.stride()):
            starts = starts[..., None] + torch.arange(n) * (s * size)
        if any(_any_on_rows(*array, starts, t.shape[-1] * size) for array in kv._arrays):
            raise ValueError("%s overlaps the cache" % name)


def _refuse_norm(out_type, x, gain, eps, residual, variant_ids, residual_out, out, scales):
    """Every check of a norm's arguments, in full; raises or returns."""
    _typed("x", x, _IN)
    _typed("gain", gain, _IN)
    if x.dim() < 1 or not x.is_contiguous():
        raise ValueError("x must be contiguous [..., d]")
    d = x.shape[-1]
    if gain.dim() not in (1, 2) or gain.shape[-1] != d or not gain.is_contiguous():
        raise ValueError("gain must be contiguous [d] or [num_gains, d] with d=%d (got %s)" % (d, tuple(gain.shape)))
    num_gains = 1 if gain.dim() == 1 else gain.shape[0]
    if d < 8 or d % 8 or d > 65536 or num_gains < 1:
        raise ValueError("d must be a multiple of 8, 8..65536, and there must be a gain (got d=%d, %d gains)"
                         % (d, num_gains))
    if not eps >= 0.0:
        raise ValueError("eps must be >= 0 (got %r)" % eps)
    lead = x.shape[:-1]
    if variant_ids is not None:
        _plain("variant_ids", variant_ids, torch.int32, lead)
    if residual is not None:
        _typed("residual", residual, _IN)
        _plain("residual", residual, residual.dtype, x.shape)
        if residual_out is not None and residual_out is not residual:
            _plain("residual_out", residual_out, residual.dtype, x.shape)
    elif residual_out is not None:
        raise ValueError("residual_out needs a residual")
    if out is not None:
        _plain("out", out, torch.bfloat16 if out_type == BD_BF16 else torch.float8_e4m3fn, x.shape)
    if scales is not None:
        _plain("scales", scales, torch.uint8, (*lead, (d + 31) // 32))
    every = [("x", x), ("gain", gain), ("residual", residual), ("variant_ids", variant_ids),
             ("residual_out", residual_out), ("out", out), ("scales", scales)]
    _same_gpu(x.device, every)
    # no output may meet anything else, but for a residual updated in place
    every = [(name, t) for name, t in every if t is not None and t.numel()]
    for name, t in every[::-1]:
        if name not in ("residual_out", "out", "scales"):
            continue
        for other, o in every:
            if other == name or (name == "residual_out" and other == "residual" and o.data_ptr() == t.data_ptr()):
                continue
            if other == "residual" and residual_out is not None and o.data_ptr() == residual_out.data_ptr():
                continue  # seen as residual_out
            if _overlap(t, o):
                raise ValueError("%s overlaps %s" % (name, other))


def _rms_norm(out_type, x, gain, eps, residual, variant_ids, residual_out, out, scales):
    eps = float(eps)
    # the ordinary call, seen through in a few comparisons; any other takes the checks one by one
    try:
        shape = x.shape
        d, dev = shape[-1], x.get_device()
        lead = shape[:-1]
        num_gains, gain_d = gain.shape
        x_type, gain_type = _IN[x.dtype], _IN[gain.dtype]
        res_type = _IN[residual.dtype] if residual is not None else BD_BF16
        ok = (dev >= 0 and 8 <= d <= 65536 and d % 8 == 0 and eps >= 0.0 and gain_d == d and num_gains >= 1
              and scales is None and x.is_contiguous() and gain.is_contiguous() and gain.get_device() == dev
              and (residual is None or (residual.shape == shape and residual.is_contiguous()
                                        and residual.get_device() == dev))
              and (variant_ids is None or (variant_ids.shape == lead and variant_ids.dtype is _INT
                                           and variant_ids.is_contiguous() and variant_ids.get_device() == dev)))
        if ok and (out is not None or residual_out is not None):
            # given outputs: of the right kind, and no two tensors meet (but for a residual updated in place)
            used = [x, gain] if variant_ids is None else [x, gain, variant_ids]
            if residual is not None:
                used.append(residual)
            if residual_out is not None and residual_out is not residual:
                ok = (residual is not None and residual_out.shape == shape and residual_out.dtype == residual.dtype
                      and residual_out.is_contiguous() and residual_out.get_device() == dev)
                used.append(residual_out)
            if out is not None:
                ok = (ok and out.shape == shape and out.is_contiguous() and out.get_device() == dev
                      and out.dtype == (torch.bfloat16 if out_type == BD_BF16 else torch.float8_e4m3fn))
                used.append(out)
            at = sorted([(t.data_ptr(), t.nbytes) for t in used])
            ok = ok and all(p + n <= q for (p, n), (q, _) in zip(at, at[1:]))
    except (AttributeError, IndexError, KeyError, TypeError, ValueError):
        ok = False
    if not ok:
        _refuse_norm(out_type, x, gain, eps, residual, variant_ids, residual_out, out, scales)
        num_gains = gain.shape[0] if gain.dim() == 2 else 1
        x_type, gain_type = _IN[x.dtype], _IN[gain.dtype]
        res_type = _IN[residual.dtype] if residual is not None else BD_BF16
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return _rms_norm(out_type, x, gain, eps, residual, variant_ids, residual_out, out, scales)
    lib = _declared or _library()
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(residual)
    if out is None:
        if out_type != BD_BF16:
            out = torch.empty(shape, dtype=torch.float8_e4m3fn, device=x.device)
        elif x_type == BD_BF16:
            out = torch.empty_like(x)
        elif residual is not None and res_type == BD_BF16:
            out = torch.empty_like(residual)
        else:
            out = torch.empty(shape, dtype=torch.bfloat16, device=x.device)
    if out_type != BD_BF16 and scales is None:
        scales = torch.empty((*lead, (d + 31) // 32), dtype=torch.uint8, device=x.device)
    st = lib.bd_rms_norm(x.data_ptr(), x_type, residual.data_ptr() if residual is not None else None,
                         residual_out.data_ptr() if residual is not None else None, res_type, gain.data_ptr(),
                         gain_type, num_gains, variant_ids.data_ptr() if variant_ids is not None else None, eps,
                         out.data_ptr(), out_type, scales.data_ptr() if scales is not None else None, x.numel() // d,
                         d, _stream_of(dev))
    if st:
        _check(lib, "bd_rms_norm", st)
    return out, scales, residual_out


def bd_rms_norm(x: torch.Tensor, gain: torch.Tensor, eps: float = 1e-5, residual: torch.Tensor | None = None,
                variant_ids: torch.Tensor | None = None, residual_out: torch.Tensor | None = None,
                out: torch.Tensor | None = None):
    """h = x + residual (kept in the residual's type); y = h / sqrt(mean(h²) + eps) · gain, as bf16.

    x [..., d] is bf16 or fp32, gain [d] or, with variant_ids (int32 [...]), [num_gains, d]: each token takes its
    variant's.  Returns y, or (y, residual_out) with a residual; residual_out may be the residual itself (updated in
    place) and is allocated where it is not given."""
    out, _, res = _rms_norm(BD_BF16, x, gain, eps, residual, variant_ids, residual_out, out, None)
    return out if residual is None else (out, res)


def bd_rms_norm_e4m3(x: torch.Tensor, gain: torch.Tensor, eps: float = 1e-5, residual: torch.Tensor | None = None,
                     variant_ids: torch.Tensor | None = None, residual_out: torch.Tensor | None = None,
                     out: torch.Tensor | None = None, scales: torch.Tensor | None = None):
    """bd_rms_norm with y held in 8 bits: (codes float8_e4m3fn [..., d], scales uint8 [..., ceil(d/32)]), one scale
    2^(byte − 127) per 32 columns, and residual_out after them with a residual."""
    out, scales, res = _rms_norm(BD_E4M3, x, gain, eps, residual, variant_ids, residual_out, out, scales)
    return (out, scales) if residual is None else (out, scales, res)


class bd_kv_cache:
    """A paged key-value cache over the caller's tensors.

    k, v: [num_pages, num_heads, page_size, head_dim], bf16 or float8_e4m3fn, alike in shape, dtype and strides,
    head_dim contiguous (a [num_pages, page_size, num_heads, head_dim] buffer goes in as its transpose(1, 2)); for 4
    bits float4_e2m1fn_x2 [num_pages, num_heads, page_size, head_dim / 2], two codes to a byte.
    k_scales, v_scales: for float8_e4m3fn uint8 [num_pages, num_heads, page_size], one scale byte per row; for
    float4_e2m1fn_x2 uint8 [num_pages, num_heads, head_dim / 32, page_size], one per 32 columns of a row.
    The tensors are kept by reference; the checks run once, here."""

    _bounds = _arrays = ()

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scales: torch.Tensor | None = None,
                 v_scales: torch.Tensor | None = None):
        kind = _typed("k", k, _HELD)
        _tensor("v", v)
        if k.dim() != 4 or v.shape != k.shape or v.dtype != k.dtype or v.stride() != k.stride():
            raise ValueError("k and v must be alike: [num_pages, num_heads, page_size, head_dim], one dtype, "
                             "one layout")
        pages, heads, page, row = k.shape
        dim = 2 * row if kind == BD_E2M1 else row
        if pages < 1 or not 1 <= heads <= 65535 or page % 8 or not 8 <= page <= 4096:
            raise ValueError("need pages, 1..65535 heads and a page size that is a multiple of 8, 8..4096 (got %s)"
                             % (tuple(k.shape),))
        least = 32 if kind == BD_E2M1 else 16
        if dim % least or not 16 <= dim <= 256:
            raise ValueError("head_dim must be a multiple of %d, %d..256 (got %d)" % (least, least, dim))
        if pages * page > 2 ** 31 - 1:
            raise ValueError("more than 2^31 - 1 slots")
        stride = list(k.stride())
        for i, n in enumerate(k.shape):
            if n == 1:
                stride[i] = 0 if i < 3 else 1  # never stepped over
        if stride[3] != 1:
            raise ValueError("head_dim must be contiguous")
        size = k.element_size()
        if any(s * size % 16 for s in stride[:3]) or k.data_ptr() % 16 or v.data_ptr() % 16:
            raise ValueError("k, v and their strides must be multiples of 16 bytes")
        # distinct rows must not overlap: each axis steps over all of the smaller ones
        steps = sorted((s, n) for s, n in zip(stride[:3], k.shape[:3]) if n > 1)
        extent = row
        for s, n in steps:
            if s < extent:
                raise ValueError("rows of k overlap (strides %s)" % (tuple(k.stride()),))
            extent = s * (n - 1) + extent
        self._span = extent * size
        if kind != BD_BF16:
            held = (pages, heads, page) if kind == BD_E4M3 else (pages, heads, dim // 32, page)
            for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
                _plain(name, t, torch.uint8, held)
                if t.data_ptr() % 8:
                    raise ValueError("%s must be 8-byte aligned" % name)
        elif k_scales is not None or v_scales is not None:
            raise ValueError("a bf16 cache has no scales")
        # where the arrays are: each as _on_rows takes it, and the ends of their spans in rising order, those that meet
        # taken together
        row, steps = row * size, [(s * size, n) for s, n in reversed(steps)]
        self._arrays = [(k.data_ptr(), steps, row), (v.data_ptr(), steps, row)]
        spans = [(at, at + self._span) for at, _, _ in self._arrays]
        if kind != BD_BF16:
            for t in (k_scales, v_scales):
                self._arrays.append((t.data_ptr(), [], t.nbytes))
                spans.append((t.data_ptr(), t.data_ptr() + t.nbytes))
        bounds = []
        for lo, hi in sorted(spans):
            if bounds and lo <= bounds[-1]:
                bounds[-1] = max(bounds[-1], hi)
            else:
                bounds += [lo, hi]
        self._bounds = bounds
        if kind != BD_BF16 and len(bounds) < 8:
            if _overlap(k_scales, v_scales):
                raise ValueError("k_scales overlaps v_scales")
            for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
                for other, rows in (("k", k), ("v", v)):
                    if _on_rows(rows.data_ptr(), steps, row, *_span(t)):
                        raise ValueError("%s overlaps %s" % (name, other))
        _same_gpu(k.device, (("v", v), ("k_scales", k_scales), ("v_scales", v_scales)))
        if abs(k.data_ptr() - v.data_ptr()) < self._span and not self._interleaved(k, v, stride, size):
            raise ValueError("k and v overlap")
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.num_pages, self.num_heads, self.page_size, self.head_dim = pages, heads, page, dim
        self.device, self._dev = k.device, k.get_device()
        self._desc = _KV(k.data_ptr(), v.data_ptr(), _at(k_scales), _at(v_scales), kind, heads, dim, page, pages,
                         *stride[:3])
        self._ref = ctypes.addressof(self._desc)

    @staticmethod
    def _interleaved(k, v, stride, size):
        """Whether v's rows lie in the gaps of k's: both are slices of one buffer, along an axis whose step leaves
        room for the other's block."""
        gap = abs(k.data_ptr() - v.data_ptr()) // size
        inner = [(s, n) for s, n in zip(stride[:3], k.shape[:3]) if n > 1 and s <= gap]
        outer = [s for s, n in zip(stride[:3], k.shape[:3]) if n > 1 and s > gap]
        block = sum(s * (n - 1) for s, n in inner) + k.shape[3]
        return block <= gap and all(gap + block <= s for s in outer)

    @classmethod
    def empty(cls, num_pages: int, num_heads: int, page_size: int, head_dim: int, dtype: torch.dtype = torch.bfloat16,
              device="cuda"):
        """A cache of its own memory, contents undefined."""
        lead, row, held = (num_pages, num_heads, page_size), head_dim, (num_pages, num_heads, page_size)
        if dtype == torch.float4_e2m1fn_x2:
            if head_dim % 32:
                raise ValueError("head_dim must be a multiple of 32 (got %d)" % head_dim)
            row, held = head_dim // 2, (num_pages, num_heads, head_dim // 32, page_size)
        k, v = (torch.empty((*lead, row), dtype=dtype, device=device) for _ in range(2))
        if dtype not in (torch.float8_e4m3fn, torch.float4_e2m1fn_x2):
            return cls(k, v)
        return cls(k, v, *(torch.empty(held, dtype=torch.uint8, device=device) for _ in range(2)))


def _rows(name, t, kv_heads, dim):
    """(type, strides, n, heads, elements from the first to behind the last) of [n, heads, dim] rows with any token and
    head stride."""
    try:
        n, heads, last = t.shape
        a, b, c = t.stride()
        kind = _IN[t.dtype]
        if last == dim and (heads == kv_heads or kv_heads is None) and c == 1 and n > 1 and heads > 1:
            unit = 7 if kind == BD_BF16 else 3   # elements of 16 bytes, less one
            if not (a | b) & unit and not t.data_ptr() & 15:
                return kind, _Pair(a, b), n, heads, (n - 1) * a + (heads - 1) * b + dim
    except (AttributeError, KeyError, ValueError):
        pass
    kind = _typed(name, t, _IN)
    if t.dim() != 3 or (kv_heads is not None and t.shape[1] != kv_heads) or t.shape[2] != dim:
        raise ValueError("%s must be [n, %s, %d] (got %s)" % (name, kv_heads or "num_q_heads", dim, tuple(t.shape)))
    (n, heads, _), (a, b, c) = t.shape, t.stride()
    if n <= 1:
        a = 0
    if heads <= 1:
        b = 0
    if c != 1:
        raise ValueError("%s's rows must be contiguous" % name)
    size = t.element_size()
    if a * size % 16 or b * size % 16 or t.data_ptr() % 16:
        raise ValueError("%s and its strides must be multiples of 16 bytes" % name)
    return kind, _Pair(a, b), n, heads, (n - 1) * a + (heads - 1) * b + dim


def _cache(kv):
    if not isinstance(kv, bd_kv_cache):
        raise TypeError("kv must be a bd_kv_cache")


def _index(name, t, n, dev):
    """Whether t is an int32 [n] index on the device, as it nearly always is."""
    return (type(t) is torch.Tensor and t.dtype is _INT and t.shape == (n,) and t.is_contiguous()
            and t.get_device() == dev)


def bd_kv_write(kv: bd_kv_cache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor):
    """Writes the rows k, v [T, num_heads, head_dim] (bf16 or fp32, any token and head strides) of T tokens into the
    cache's slots (int32 [T]; slot = page · page_size + place).  Slots below 0 or past the cache's end are skipped; of
    several tokens with one slot the last stays.  k, v and slots lie apart from the cache's rows (copy a view of them
    first to move rows within one)."""
    _cache(kv)
    kind, ks, T, _, k_reach = _rows("k", k, kv.num_heads, kv.head_dim)
    v_kind, vs, v_n, _, v_reach = _rows("v", v, kv.num_heads, kv.head_dim)
    dev = kv._dev
    if v_kind != kind or v_n != T:
        raise ValueError("k and v must have one dtype and one number of tokens")
    # the ordinary call: k, v and all between them (one q, k, v result, mostly) and slots outside the cache's spans
    k0, v0, size, ends = k.data_ptr(), v.data_ptr(), _SIZE[kind], kv._bounds
    at = bisect_right(ends, k0 if k0 < v0 else v0)
    upto = ends[at] if at < len(ends) else _NO_END
    if not (_index("slots", slots, T, dev) and k.get_device() == dev and v.get_device() == dev
            and (not at & 1 and k0 + size * k_reach <= upto and v0 + size * v_reach <= upto
                 or _apart(kv, k0, k0 + size * k_reach) and _apart(kv, v0, v0 + size * v_reach))
            and _apart(kv, slots.data_ptr(), slots.data_ptr() + 4 * T)):
        _plain("slots", slots, torch.int32, (T,))
        _refuse_on_cache(kv, (("k", k), ("v", v), ("slots", slots)))
        _same_gpu(kv.device, (("k", k), ("v", v), ("slots", slots)))
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return bd_kv_write(kv, k, v, slots)
    lib = _declared or _library()
    st = lib.bd_kv_write(kv._ref, k0, ks, v0, vs, kind, slots.data_ptr(), T, _stream_of(dev))
    if st:
        _check(lib, "bd_kv_write", st)


def _given(t, dtype, shape, dev):
    """Whether t is a contiguous tensor of this kind on the device."""
    return (type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and t.get_device() == dev)


def _read_to(kv, out, slots, shape, dev):
    """Whether out is two tensors that a read may write to, as it nearly always is."""
    if type(out) not in (tuple, list) or len(out) != 2:
        return False
    k, v = out
    if not (_given(k, torch.bfloat16, shape, dev) and _given(v, torch.bfloat16, shape, dev)):
        return False
    k0, v0, s0, size = k.data_ptr(), v.data_ptr(), slots.data_ptr(), k.nbytes
    k1, v1, s1 = k0 + size, v0 + size, s0 + slots.nbytes
    return ((k1 <= v0 or v1 <= k0) and (k1 <= s0 or s1 <= k0) and (v1 <= s0 or s1 <= v0) and _apart(kv, k0, k1)
            and _apart(kv, v0, v1))


def bd_kv_read(kv: bd_kv_cache, slots: torch.Tensor, out: tuple[torch.Tensor, torch.Tensor] | None = None):
    """The rows of T slots (int32 [T]) as bf16 (k, v), each [T, num_heads, head_dim], exactly as held.  Slots below 0
    give zeros, slots past the cache's end NaN.  out, if given, lies apart from the cache's rows and from slots."""
    _cache(kv)
    _tensor("slots", slots)
    dev, n = kv._dev, slots.numel()
    shape = (n, kv.num_heads, kv.head_dim)
    if not (_index("slots", slots, n, dev) and (out is None or _read_to(kv, out, slots, shape, dev))):
        _plain("slots", slots, torch.int32, shape[:1])
        given = [] if out is None else list(zip(("out[0]", "out[1]"), out, strict=True))
        for name, t in given:
            _plain(name, t, torch.bfloat16, shape)
        if given and n and _overlap(*out):
            raise ValueError("out[0] overlaps out[1]")
        for name, t in given:
            if n and _overlap(t, slots):
                raise ValueError("%s overlaps slots" % name)
        _refuse_on_cache(kv, given)
        _same_gpu(kv.device, [("slots", slots)] + given)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return bd_kv_read(kv, slots, out)
    lib = _declared or _library()
    if out is None:
        k = torch.empty(shape, dtype=torch.bfloat16, device=kv.device)
        v = torch.empty_like(k)
    else:
        k, v = out
    st = lib.bd_kv_read(kv._ref, slots.data_ptr(), n, k.data_ptr(), v.data_ptr(), _stream_of(dev))
    if st:
        _check(lib, "bd_kv_read", st)
    return k, v


def _attend_to(kv, q0, q1, page_table, lengths, out, lse, B, heads, dev, more=()):
    """Whether out and lse, as far as given, are tensors that an attention may write to, as they nearly always are: of
    the right kind, apart from each other and from all that it reads (queries from q0 up to q1)."""
    mine = []
    if out is not None:
        if not _given(out, torch.bfloat16, (B, heads, kv.head_dim), dev):
            return False
        mine.append(out)
    if lse is not None:
        if not _given(lse, torch.float32, (B, heads), dev):
            return False
        mine.append(lse)
    used = [(q0, q1)]
    for t in (page_table, lengths, *more):
        used.append((t.data_ptr(), t.data_ptr() + t.nbytes))
    for t in mine:
        lo = t.data_ptr()
        hi = lo + t.nbytes
        if not _apart(kv, lo, hi):
            return False
        for a, b in used:
            if a < hi and lo < b:
                return False
        used.append((lo, hi))
    return True


def _cap(cap):
    """A cap of scores as the library takes it."""
    if cap is None:
        return 0.0
    cap = float(cap)
    if not 2.0 ** -60 <= cap <= 2.0 ** 60:
        raise ValueError("cap must be 2^-60 .. 2^60 (got %r)" % cap)
    return cap


def _refuse_attend(q, kv, page_table, lengths, out, lse, heads, slopes=None, first=None):
    """The checks of an attention's tensors, in full; raises or returns."""
    B = q.shape[0]
    if heads < 1 or heads > 65535 or heads % kv.num_heads:
        raise ValueError("q's heads must be a multiple of the cache's %d, at most 65535 (got %d)"
                         % (kv.num_heads, heads))
    _tensor("page_table", page_table)
    if page_table.dtype != torch.int32:
        raise TypeError("page_table must be torch.int32 (got %s)" % page_table.dtype)
    if page_table.dim() != 2 or page_table.shape[0] != B or page_table.shape[1] < 1:
        raise ValueError("page_table must be [%d, max_pages] (got %s)" % (B, tuple(page_table.shape)))
    if page_table.shape[1] > 1 and page_table.stride(1) != 1:
        raise ValueError("page_table's rows must be contiguous")
    if page_table.shape[1] * kv.page_size > 1 << 24:
        raise ValueError("page_table holds more than 2^24 tokens per sequence")
    _plain("lengths", lengths, torch.int32, (B,))
    if slopes is not None:
        _plain("slopes", slopes, torch.float32, (heads,))
    if first is not None:
        _plain("first", first, torch.int32, (B,))
    if out is not None:
        _plain("out", out, torch.bfloat16, (B, heads, kv.head_dim))
    if lse is not None:
        _plain("lse", lse, torch.float32, (B, heads))
    every = (("q", q), ("page_table", page_table), ("lengths", lengths), ("slopes", slopes), ("first", first),
             ("out", out), ("lse", lse))
    given = [(name, t) for name, t in every if t is not None and t.numel()]
    for name, t in given:
        for other, o in given:
            if name in ("out", "lse") and other != name and _overlap(t, o):
                raise ValueError("%s overlaps %s" % (name, other))
    _refuse_on_cache(kv, [(name, t) for name, t in given if name in ("out", "lse")])
    _same_gpu(kv.device, every)


def bd_attend(q: torch.Tensor, kv: bd_kv_cache, page_table: torch.Tensor, lengths: torch.Tensor,
              scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
              cap: float | None = None, slopes: torch.Tensor | None = None, first: torch.Tensor | None = None):
    """softmax(scale · q kᵀ) v of one new token per sequence over the cache; bf16 [B, num_q_heads, head_dim].

    q [B, num_q_heads, head_dim] is bf16 or fp32 (any token and head strides); num_q_heads is a multiple of the cache's
    heads.  page_table int32 [B, max_pages] (rows may be strided) and lengths int32 [B] say which tokens: lengths
    counts the new one, whose row is in the cache by then.  A length of 0 gives zeros.  scale defaults to
    head_dim^-0.5.  lse, if given, is an fp32 [B, num_q_heads] tensor that receives the log of the softmax's sum.  out
    and lse lie apart from each other and from all that is read.  Where the table has room for few tokens (some
    hundreds, whatever the lengths) nothing is split and no second kernel is launched: for short sequences a table no
    wider than needed is faster.

    cap makes cap · tanh(score / cap) of the scores, slopes (fp32 [num_q_heads]) takes slopes · distance off them after
    that, and first (int32 [B]) leaves out the tokens before it: a window of w tokens has first = lengths − w.  Pages
    that hold only tokens before first need not be in the table any more."""
    _cache(kv)
    kind, qs, B, heads, reach = _rows("q", q, None, kv.head_dim)
    dev = kv._dev
    scale = kv.head_dim ** -0.5 if scale is None else float(scale)
    if not abs(scale) <= 2.0 ** 60:
        raise ValueError("scale must be at most 2^60 (got %r)" % scale)
    formed = cap is not None or slopes is not None or first is not None
    limit = _cap(cap) if formed else 0.0
    q0 = q.data_ptr()
    if not (type(page_table) is torch.Tensor and page_table.dim() == 2
            and page_table.dtype is _INT and page_table.shape[0] == B and page_table.is_contiguous()
            and 1 <= page_table.shape[1] <= (1 << 24) // kv.page_size and page_table.get_device() == dev
            and _index("lengths", lengths, B, dev) and q.get_device() == dev and 1 <= heads <= 65535
            and heads % kv.num_heads == 0
            and (not formed or (slopes is None or _given(slopes, torch.float32, (heads,), dev))
                 and (first is None or _index("first", first, B, dev)))
            and (out is None and lse is None
                 or _attend_to(kv, q0, q0 + reach * _SIZE[kind], page_table, lengths, out, lse, B, heads, dev,
                               [t for t in (slopes, first) if t is not None]))):
        _refuse_attend(q, kv, page_table, lengths, out, lse, heads, slopes, first)
    if _current_device() != dev:
        with torch.cuda.device(dev):
            return bd_attend(q, kv, page_table, lengths, scale, out, lse, cap, slopes, first)
    lib = _declared or _library()
    pages = page_table.shape[1]
    nbytes = _attend_bytes(B, heads, kv.num_heads, kv.head_dim, kv.page_size, pages)
    if out is None:
        if kind == BD_BF16 and q.is_contiguous():
            out = torch.empty_like(q)
        else:
            out = torch.empty((B, heads, kv.head_dim), dtype=torch.bfloat16, device=kv.device)
    ws = _workspace(nbytes, kv.device)
    if formed:
        scores = _Scores(limit, _at(slopes), _at(first), None)
        st = lib.bd_attend_scores(kv._ref, q0, kind, qs, heads, page_table.data_ptr(),
                                  page_table.stride(0) if B > 1 else 0, pages, lengths.data_ptr(), B, scale,
                                  ctypes.byref(scores), out.data_ptr(), _at(lse), _at(ws), nbytes, _stream_of(dev))
    else:
        st = lib.bd_attend(kv._ref, q0, kind, qs, heads, page_table.data_ptr(),
                           page_table.stride(0) if B > 1 else 0, pages, lengths.data_ptr(), B, scale, out.data_ptr(),
                           lse.data_ptr() if lse is not None else None, ws.data_ptr() if ws is not None else None, nbytes,
                           _stream_of(dev))
    if st:
        _check(lib, "bd_attend", st)
    return out


@functools.lru_cache(maxsize=4096)
def _attend_bytes(*sizes):
    """The library's answer for these sizes: a host function of nothing else."""
    return _library().bd_attend_workspace_bytes(*sizes)
