"""Refusals of the step operators (include/bitdelta_step.h): the C ABI's argument checks, which run on the host before
any HIP call, and the Python binding's, which run on host tensors."""

import ctypes

import pytest
import torch

import tenant_serving_amd as bd
from tenant_serving_amd import step

FAKE = 1 << 20          # 16-byte aligned, never dereferenced
OFF = FAKE + 2
OK, NULL, SHAPE, ALIGN, WORKSPACE, MODE = 0, 1, 2, 3, 4, 5


@pytest.fixture(scope="module")
def lib():
    return step._library()


def _kv(**change):
    d = dict(k=FAKE, v=FAKE, k_scales=FAKE, v_scales=FAKE, type=2, num_heads=2, head_dim=64, page_size=16,
             num_pages=10, page_stride=2048, head_stride=1024, token_stride=64)
    d.update(change)
    return step._KV(**d)


BAD_KV = [(dict(k=None), NULL), (dict(v=None), NULL), (dict(k_scales=None), NULL), (dict(v_scales=None), NULL),
          (dict(type=1), MODE), (dict(type=3), MODE), (dict(num_heads=0), SHAPE), (dict(num_heads=65536), SHAPE),
          (dict(head_dim=0), SHAPE), (dict(head_dim=72), SHAPE), (dict(head_dim=272), SHAPE),
          (dict(page_size=0), SHAPE), (dict(page_size=12), SHAPE), (dict(page_size=4104), SHAPE),
          (dict(num_pages=0), SHAPE), (dict(num_pages=1 << 27), SHAPE), (dict(page_stride=-16), SHAPE),
          (dict(page_stride=2056), ALIGN), (dict(head_stride=1032), ALIGN), (dict(token_stride=68), ALIGN),
          (dict(type=0, token_stride=68), ALIGN), (dict(k=OFF), ALIGN), (dict(v=OFF), ALIGN),
          (dict(k_scales=OFF), ALIGN), (dict(v_scales=OFF), ALIGN)]


def _pair(a, b):
    return step._Pair(a, b)


def test_norm_refusals(lib):
    base = dict(x=FAKE, x_type=0, residual=FAKE, residual_out=FAKE, residual_type=1, gain=FAKE, gain_type=0,
                num_gains=3, ids=FAKE, eps=1e-5, out=FAKE, out_type=2, scales=FAKE, M=4, d=64, stream=None)
    call = lambda **c: lib.bd_rms_norm(*{**base, **c}.values())  # noqa: E731
    for change, want in [(dict(x=None), NULL), (dict(gain=None), NULL), (dict(out=None), NULL),
                         (dict(scales=None), NULL), (dict(residual=None), NULL), (dict(residual_out=None), NULL),
                         (dict(x_type=2), MODE), (dict(gain_type=5), MODE), (dict(residual_type=2), MODE),
                         (dict(out_type=1), MODE), (dict(M=-1), SHAPE), (dict(d=0), SHAPE), (dict(d=60), SHAPE),
                         (dict(d=65544), SHAPE), (dict(num_gains=0), SHAPE), (dict(eps=-1.0), SHAPE),
                         (dict(eps=float("nan")), SHAPE), (dict(x=OFF), ALIGN), (dict(gain=OFF), ALIGN),
                         (dict(residual=OFF), ALIGN), (dict(residual_out=OFF), ALIGN), (dict(out=OFF), ALIGN),
                         (dict(out_type=0, out=FAKE + 8), ALIGN), (dict(ids=OFF), ALIGN)]:
        assert call(**change) == want, change
    assert call(M=0, x=None, out=None, residual=None, residual_out=None, scales=None) == OK


def test_kv_refusals(lib):
    for change, want in BAD_KV:
        kv = _kv(**change)
        r = ctypes.byref(kv)
        assert lib.bd_kv_write(r, FAKE, _pair(128, 64), FAKE, _pair(128, 64), 0, FAKE, 4, None) == want, change
        assert lib.bd_kv_read(r, FAKE, 4, FAKE, FAKE, None) == want, change
        assert lib.bd_attend(r, FAKE, 0, _pair(128, 64), 4, FAKE, 3, 3, FAKE, 2, 0.1, FAKE, None, FAKE, 1 << 30,
                             None) == want, change
    kv = _kv()
    r = ctypes.byref(kv)
    w = lambda k=FAKE, ks=_pair(128, 64), v=FAKE, vs=_pair(128, 64), t=0, s=FAKE, T=4: lib.bd_kv_write(  # noqa: E731
        r, k, ks, v, vs, t, s, T, None)
    assert lib.bd_kv_write(None, FAKE, _pair(128, 64), FAKE, _pair(128, 64), 0, FAKE, 4, None) == NULL
    assert w(k=None) == NULL and w(v=None) == NULL and w(s=None) == NULL and w(ks=None) == NULL and w(vs=None) == NULL
    assert w(t=2) == MODE and w(T=-1) == SHAPE and w(T=(1 << 28) + 1) == SHAPE
    assert w(ks=_pair(-8, 64)) == SHAPE and w(ks=_pair(132, 64)) == ALIGN and w(vs=_pair(128, 68)) == ALIGN
    assert w(t=1, ks=_pair(132, 64), vs=_pair(128, 66)) == ALIGN
    assert w(k=OFF) == ALIGN and w(v=OFF) == ALIGN and w(s=OFF) == ALIGN
    assert w(T=0, k=None, v=None, s=None) == OK
    rd = lambda s=FAKE, T=4, k=FAKE, v=FAKE: lib.bd_kv_read(r, s, T, k, v, None)  # noqa: E731
    assert rd(s=None) == NULL and rd(k=None) == NULL and rd(v=None) == NULL and rd(T=-1) == SHAPE
    assert rd(k=OFF) == ALIGN and rd(v=OFF) == ALIGN and rd(s=OFF) == ALIGN
    assert rd(T=0, s=None, k=None, v=None) == OK


def test_attend_refusals(lib):
    kv = _kv()
    need = lib.bd_attend_workspace_bytes(2, 4, 2, 64, 16, 100)
    assert need > 0
    base = dict(kv=ctypes.byref(kv), q=FAKE, q_type=0, qs=_pair(256, 64), heads=4, table=FAKE, stride=100, pages=100,
                lengths=FAKE, B=2, scale=0.125, out=FAKE, lse=FAKE, ws=FAKE, bytes=need, stream=None)
    call = lambda **c: lib.bd_attend(*{**base, **c}.values())  # noqa: E731
    for change, want in [(dict(kv=None), NULL), (dict(q=None), NULL), (dict(qs=None), NULL), (dict(table=None), NULL),
                         (dict(lengths=None), NULL), (dict(out=None), NULL), (dict(q_type=2), MODE),
                         (dict(B=-1), SHAPE), (dict(heads=0), SHAPE), (dict(heads=3), SHAPE), (dict(heads=65538), SHAPE),
                         (dict(pages=0), SHAPE), (dict(pages=(1 << 20) + 1), SHAPE), (dict(stride=-1), SHAPE),
                         (dict(scale=float("inf")), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(scale=-2.0 ** 61), SHAPE),
                         (dict(qs=_pair(-8, 64)), SHAPE), (dict(qs=_pair(260, 64)), ALIGN), (dict(q=OFF), ALIGN),
                         (dict(out=OFF), ALIGN), (dict(table=OFF), ALIGN), (dict(lengths=OFF), ALIGN),
                         (dict(lse=OFF), ALIGN), (dict(ws=None), WORKSPACE), (dict(bytes=need - 4), WORKSPACE),
                         (dict(ws=FAKE + 8), WORKSPACE), (dict(B=1 << 23), SHAPE)]:
        assert call(**change) == want, change
    assert call(B=0, q=None, table=None, lengths=None, out=None, ws=None, bytes=0) == OK


def test_workspace_query(lib):
    f = lib.bd_attend_workspace_bytes
    # a few hundred tokens at most: nothing is split
    assert f(2, 4, 2, 64, 16, 8) == f(2, 4, 2, 64, 16, 24) == f(2, 4, 2, 256, 16, 24) == f(512, 4, 2, 256, 16, 64) == 0
    # two places for each workgroup, of 16 heads' sums, maxima and outputs; workgroups for every unit at most
    place = 16 * 66 * 4
    assert 4 * 13 * 2 * place <= f(2, 4, 2, 64, 16, 100) <= 4 * (13 + 2) * 2 * place + 4096
    assert f(512, 4, 2, 256, 16, 65) > 0 and f(2, 4, 2, 256, 16, 25) > 0
    assert f(256, 6, 3, 256, 16, 128) == 0 and f(256, 6, 3, 256, 16, 129) > 0
    assert f(64, 64, 8, 128, 16, 1024) == f(128, 64, 8, 128, 16, 1024)   # no more than the GPU's workgroups
    for bad in [(0, 4, 2, 64, 16, 9), (2, 3, 2, 64, 16, 9), (2, 4, 0, 64, 16, 9), (2, 4, 2, 72, 16, 9),
                (2, 4, 2, 64, 12, 9), (2, 4, 2, 64, 16, 0), (2, 4, 2, 64, 16, 1 << 21)]:
        assert f(*bad) == 0


# ----------------------------------------------------------------------------
# the Python binding

def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_binding_norm_refusals():
    x, g = _t(5, 64), _t(3, 64)
    ids = _t(5, dtype=torch.int32)
    for err, match, args, kw in [
            (TypeError, "x must be", (x.double(), g), {}), (TypeError, "x must be", (None, g), {}),
            (TypeError, "gain", (x, g.half()), {}), (ValueError, "gain", (x, _t(3, 72)), {}),
            (ValueError, "contiguous", (_t(64, 5).t(), g), {}), (ValueError, "multiple of 8", (_t(5, 60), _t(3, 60)), {}),
            (ValueError, "multiple of 8", (_t(5, 65544), _t(1, 65544)), {}), (ValueError, "eps", (x, g, -1.0), {}),
            (ValueError, "variant_ids", (x, g), dict(variant_ids=ids[:4])),
            (TypeError, "variant_ids", (x, g), dict(variant_ids=ids.long())),
            (ValueError, "residual", (x, g), dict(residual=_t(4, 64))),
            (TypeError, "residual", (x, g), dict(residual=x.half())),
            (ValueError, "needs a residual", (x, g), dict(residual_out=x)),
            (TypeError, "residual_out", (x, g), dict(residual=x, residual_out=x.float())),
            (TypeError, "out", (x, g), dict(out=x.float())), (ValueError, "out", (x, g), dict(out=_t(4, 64))),
            (ValueError, "GPU", (x, g), {})]:
        with pytest.raises(err, match=match):
            bd.bd_rms_norm(*args, **kw)
    with pytest.raises(TypeError, match="out"):
        bd.bd_rms_norm_e4m3(x, g, out=_t(5, 64))
    with pytest.raises(ValueError, match="scales"):
        bd.bd_rms_norm_e4m3(x, g, scales=_t(5, 3, dtype=torch.uint8))


def test_binding_cache_refusals():
    k = _t(6, 2, 16, 64)
    s = _t(6, 2, 16, dtype=torch.uint8)
    k8 = k.to(torch.float8_e4m3fn)
    for err, match, args in [
            (TypeError, "k must be", (k.half(), k.half())), (ValueError, "alike", (k, _t(6, 2, 16, 80))),
            (ValueError, "alike", (k, k8)), (ValueError, "alike", (k[0], k[0])),
            (ValueError, "page size", (_t(6, 2, 12, 64),) * 2), (ValueError, "page size", (_t(0, 2, 16, 64),) * 2),
            (ValueError, "head_dim", (_t(6, 2, 16, 72),) * 2), (ValueError, "head_dim", (_t(6, 2, 16, 272),) * 2),
            (ValueError, "contiguous", (_t(6, 2, 64, 16).transpose(2, 3),) * 2),
            (ValueError, "16 bytes", (_t(6, 2, 16, 68)[..., :64],) * 2),
            (ValueError, "overlap", (_t(1, 2, 16, 64).expand(6, 2, 16, 64),) * 2),
            (ValueError, "no scales", (k, k.clone(), s, s)), (TypeError, "k_scales", (k8, k8.clone())),
            (ValueError, "k_scales", (k8, k8.clone(), s[:5], s)), (ValueError, "GPU", (k, k.clone()))]:
        with pytest.raises(err, match=match):
            bd.bd_kv_cache(*args)
    # slices of one buffer that do not meet pass the layout checks (and are refused for the device)
    both = _t(6, 2, 2, 16, 64)
    with pytest.raises(ValueError, match="GPU"):
        bd.bd_kv_cache(both[:, 0], both[:, 1])
    both = _t(6, 16, 2, 2, 64)
    with pytest.raises(ValueError, match="GPU"):
        bd.bd_kv_cache(both[:, :, 0].transpose(1, 2), both[:, :, 1].transpose(1, 2))


def _pretend():
    """What the calls' checks read of a bd_kv_cache, on the host."""
    kv = object.__new__(bd.bd_kv_cache)
    kv.num_pages, kv.num_heads, kv.page_size, kv.head_dim = 6, 2, 16, 64
    kv.device, kv._dev = torch.device("cpu"), 0
    return kv


def test_interleaved_slices():
    f = bd.bd_kv_cache._interleaved
    both = _t(6, 2, 2, 16, 64)
    k, v = both[:, 0], both[:, 1]
    assert f(k, v, list(k.stride()), 2)
    k, v = both[:, 0], both[:, 0, :, 1:]     # one token further on: rows meet
    assert not f(k, v, list(k.stride()), 2)
    k = _t(6, 2, 16, 64)
    assert not f(k, k, list(k.stride()), 2)


def test_binding_call_refusals():
    kv = _pretend()
    k, slots = _t(4, 2, 64), _t(4, dtype=torch.int32)
    for err, match, args in [
            (TypeError, "bd_kv_cache", (None, k, k, slots)), (TypeError, "k must be", (kv, k.half(), k, slots)),
            (ValueError, "k must be", (kv, _t(4, 3, 64), k, slots)), (ValueError, "v must be", (kv, k, _t(4, 2, 80), slots)),
            (ValueError, "one dtype", (kv, k, k.float(), slots)), (ValueError, "one dtype", (kv, k, _t(5, 2, 64), slots)),
            (ValueError, "contiguous", (kv, _t(4, 64, 2).transpose(1, 2), k, slots)),
            (ValueError, "16 bytes", (kv, _t(4, 2, 68)[..., :64], k, slots)),
            (ValueError, "slots", (kv, k, k, slots[:3])), (TypeError, "slots", (kv, k, k, slots.long())),
            (ValueError, "GPU", (kv, k, k, slots))]:
        with pytest.raises(err, match=match):
            bd.bd_kv_write(*args)
    with pytest.raises(TypeError, match="slots"):
        bd.bd_kv_read(kv, slots.long())
    with pytest.raises(ValueError, match="out"):
        bd.bd_kv_read(kv, slots, out=(k[:3], k))
    with pytest.raises(ValueError, match="overlaps"):
        bd.bd_kv_read(kv, slots, out=(k, k))
    with pytest.raises(ValueError, match="GPU"):
        bd.bd_kv_read(kv, slots)
    q, table, lens = _t(3, 4, 64), _t(3, 5, dtype=torch.int32), _t(3, dtype=torch.int32)
    for err, match, args, kw in [
            (TypeError, "bd_kv_cache", (q, None, table, lens), {}), (TypeError, "q must be", (q.half(), kv, table, lens), {}),
            (ValueError, "q must be", (_t(3, 4, 80), kv, table, lens), {}),
            (ValueError, "multiple of the cache", (_t(3, 3, 64), kv, table, lens), {}),
            (TypeError, "page_table", (q, kv, table.long(), lens), {}),
            (ValueError, "page_table", (q, kv, table[:2], lens), {}), (ValueError, "page_table", (q, kv, table[:, :0], lens), {}),
            (ValueError, "page_table", (q, kv, _t(5, 3, dtype=torch.int32).t(), lens), {}),
            (ValueError, "2\\^24", (q, kv, torch.zeros(((1 << 20) + 1,), dtype=torch.int32).as_strided((3, (1 << 20) + 1), (0, 1)), lens), {}),
            (ValueError, "lengths", (q, kv, table, lens[:2]), {}), (TypeError, "lengths", (q, kv, table, lens.long()), {}),
            (ValueError, "scale", (q, kv, table, lens, float("nan")), {}),
            (ValueError, "out", (q, kv, table, lens), dict(out=_t(3, 5, 64))),
            (TypeError, "out", (q, kv, table, lens), dict(out=q.float())),
            (TypeError, "lse", (q, kv, table, lens), dict(lse=_t(3, 4))), (ValueError, "GPU", (q, kv, table, lens), {})]:
        with pytest.raises(err, match=match):
            bd.bd_attend(*args, **kw)
