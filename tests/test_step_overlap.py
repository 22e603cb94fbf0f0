"""Refusals of the step operators where an output's memory meets something else (include/bitdelta_step.h says what has
to lie apart): the binding's checks, on host tensors."""

import pytest
import torch

import tenant_serving_amd as bd

BF, E4 = torch.bfloat16, torch.float8_e4m3fn


def test_scales_apart_from_each_other_and_from_the_codes():
    k, v = (torch.zeros((6, 2, 16, 64), dtype=torch.uint8).view(E4) for _ in range(2))
    n = 6 * 2 * 16
    s = torch.zeros(3 * n, dtype=torch.uint8)
    one = s[:n].view(6, 2, 16)
    for a, b, match in ((one, one, "k_scales overlaps v_scales"),
                        (one, s[n - 8:2 * n - 8].view(6, 2, 16), "k_scales overlaps v_scales"),
                        (s[n - 8:2 * n - 8].view(6, 2, 16), one, "k_scales overlaps v_scales"),
                        (k.view(torch.uint8).view(-1)[128:128 + n].view(6, 2, 16), one, "k_scales overlaps k"),
                        (one, v.view(torch.uint8).view(-1)[-n:].view(6, 2, 16), "v_scales overlaps v"),
                        (one, k.view(torch.uint8).view(-1)[:n].view(6, 2, 16), "v_scales overlaps k"),
                        (one, s[n:2 * n].view(6, 2, 16), "GPU")):
        with pytest.raises(ValueError, match=match):
            bd.bd_kv_cache(k, v, a, b)
    # one allocation of pages with room behind each row's codes: the scales may lie between rows, not on them
    wide = torch.zeros((2, 2, 16, 256), dtype=torch.uint8)
    k, v = wide[:1, :, :, :64].view(E4), wide[1:, :, :, :64].view(E4)
    row = wide[0, 0, 0]
    with pytest.raises(ValueError, match="GPU"):
        bd.bd_kv_cache(k, v, row[64:96].view(1, 2, 16), row[96:128].view(1, 2, 16))
    with pytest.raises(ValueError, match="k_scales overlaps k"):
        bd.bd_kv_cache(k, v, row[56:88].view(1, 2, 16), row[96:128].view(1, 2, 16))
    with pytest.raises(ValueError, match="v_scales overlaps k"):
        bd.bd_kv_cache(k, v, row[64:96].view(1, 2, 16), row[232:].as_strided((1, 2, 16), (32, 16, 1)))


def _cache(monkeypatch, k, v, *scales):
    """A bd_kv_cache over host tensors, for its calls' checks: the calls go as far as to refuse the device."""
    from tenant_serving_amd import step
    with monkeypatch.context() as m:
        m.setattr(step, "_same_gpu", lambda device, named: None)
        kv = bd.bd_kv_cache(k, v, *scales)
    kv._dev = 0
    return kv


def test_written_rows_apart_from_the_cache(monkeypatch):
    k, v = (torch.zeros((6, 2, 16, 64), dtype=BF) for _ in range(2))
    kv = _cache(monkeypatch, k, v)
    rows, slots = torch.zeros((16, 2, 64), dtype=BF), torch.zeros(16, dtype=torch.int32)
    page = k[1].transpose(0, 1)                          # a page's rows, as a copy to another page would take them
    for args, match in (((page, rows, slots), "k overlaps the cache"), ((rows, v[2].transpose(0, 1), slots), "v overlaps the cache"),
                        ((k[1, :, :1].transpose(0, 1), rows[:1], slots[:1]), "k overlaps the cache"),
                        ((rows, rows, k.view(torch.int32).view(-1)[32:48]), "slots overlaps the cache"),
                        ((rows.float(), rows.float(), v.view(torch.int32).view(-1)[-16:]), "slots overlaps the cache"),
                        ((rows, rows, slots), "GPU")):
        with pytest.raises(ValueError, match=match):
            bd.bd_kv_write(kv, *args)
    s = [torch.zeros((6, 2, 16), dtype=torch.uint8) for _ in range(2)]
    k8, v8 = (torch.zeros((6, 2, 16, 64), dtype=torch.uint8).view(E4) for _ in range(2))
    kv = _cache(monkeypatch, k8, v8, *s)
    for t in (*s, k8.view(torch.uint8), v8.view(torch.uint8)):
        with pytest.raises(ValueError, match="slots overlaps the cache"):
            bd.bd_kv_write(kv, rows, rows, t.view(-1).view(torch.int32)[-16:])
    with pytest.raises(ValueError, match="GPU"):
        bd.bd_kv_write(kv, rows, rows, slots)


def test_written_rows_in_the_gaps_of_the_cache(monkeypatch):
    """Rows between the cache's own, in one buffer with them, are apart from it: another layer's, for one."""
    both = torch.zeros((6, 2, 2, 2, 16, 64), dtype=BF)   # pages, layers, keys and values, heads, places, dim
    kv = _cache(monkeypatch, both[:, 0, 0], both[:, 0, 1])
    slots = torch.zeros(16, dtype=torch.int32)
    other = both[3, 1, 0].transpose(0, 1), both[3, 1, 1].transpose(0, 1)
    with pytest.raises(ValueError, match="GPU"):
        bd.bd_kv_write(kv, *other, slots)
    with pytest.raises(ValueError, match="v overlaps the cache"):
        bd.bd_kv_write(kv, other[0], both[3, 0, 1].transpose(0, 1), slots)
    # tokens six buffers apart, each with its rows in another layer's pages, and one of them in this one's
    far = both[:, 1, 0, :, 5]
    with pytest.raises(ValueError, match="GPU"):
        bd.bd_kv_write(kv, far, far, slots[:6])
    with pytest.raises(ValueError, match="k overlaps the cache"):
        bd.bd_kv_write(kv, both[:, 0, 1, :, 5], far, slots[:6])
    # rows that begin in a gap and end on the cache's
    flat = both.view(-1)
    cut = flat[2 * 2048 - 32:].as_strided((3, 2, 64), (8192, 1024, 1))
    with pytest.raises(ValueError, match="GPU"):
        bd.bd_kv_write(kv, flat[2 * 2048:].as_strided((3, 2, 64), (8192, 1024, 1)), far[:3], slots[:3])
    with pytest.raises(ValueError, match="k overlaps the cache"):
        bd.bd_kv_write(kv, cut, far[:3], slots[:3])


def test_rows_read_back_apart_from_the_cache_and_the_slots(monkeypatch):
    k, v = (torch.zeros((6, 2, 16, 64), dtype=BF) for _ in range(2))
    slots = torch.zeros(16, dtype=torch.int32)
    out = [torch.zeros((16, 2, 64), dtype=BF) for _ in range(2)]
    kv = _cache(monkeypatch, k, v)
    rows = k.view(-1)[2048:4096].view(16, 2, 64)
    for a, b, match in ((rows, out[1], r"out\[0\] overlaps the cache"), (out[0], v.view(-1)[:2048].view(16, 2, 64), r"out\[1\] overlaps the cache"),
                        (out[0], out[1], "GPU")):
        with pytest.raises(ValueError, match=match):
            bd.bd_kv_read(kv, slots, out=(a, b))
    with pytest.raises(ValueError, match=r"out\[1\] overlaps slots"):
        bd.bd_kv_read(kv, out[1].view(torch.int32).view(-1)[-16:], out=out)
    s = [torch.zeros(16 * 2 * 64 * 2, dtype=torch.uint8) for _ in range(2)]
    k8, v8 = (torch.zeros((6, 2, 16, 64), dtype=torch.uint8).view(E4) for _ in range(2))
    kv = _cache(monkeypatch, k8, v8, *(t[-192:].view(6, 2, 16) for t in s))
    for i in (0, 1):
        with pytest.raises(ValueError, match=r"out\[0\] overlaps the cache"):
            bd.bd_kv_read(kv, slots, out=(s[i].view(BF).view(16, 2, 64), out[1]))
    # in the gaps of the cache's strides
    both = torch.zeros((6, 2, 2, 16, 64), dtype=BF)
    kv = _cache(monkeypatch, both[:, 0], torch.zeros_like(both)[:, 0])
    with pytest.raises(ValueError, match="GPU"):
        bd.bd_kv_read(kv, slots, out=(both[2, 1].view(16, 2, 64), out[1]))
    with pytest.raises(ValueError, match="overlaps the cache"):
        bd.bd_kv_read(kv, slots, out=(both[2, 0].view(16, 2, 64), out[1]))
