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
    for args, match in (((page, rows, slots), "k overlaps the cache"),
                        ((rows, v[2].transpose(0, 1), slots), "v overlaps the cache"),
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
    for a, b, match in ((rows, out[1], r"out\[0\] overlaps the cache"),
                        (out[0], v.view(-1)[:2048].view(16, 2, 64), r"out\[1\] overlaps the cache"),
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


def test_attention_outputs_apart_from_all_it_reads(monkeypatch):
    """The same answer with and without lse, and for either output."""
    both = [torch.zeros((6, 2, 2, 16, 64), dtype=BF) for _ in range(2)]
    kv = _cache(monkeypatch, both[0][:, 0], both[1][:, 0])
    q = torch.zeros((16, 4, 64), dtype=BF)
    table, lens = torch.zeros((16, 2048), dtype=torch.int32), torch.zeros(2048, dtype=torch.int32)[:16]
    fine, lse = torch.zeros((16, 4, 64), dtype=BF), torch.zeros((16, 4))
    on_lens = lens.as_strided((2048,), (1,)).view(BF).view(-1)[:4096].view(16, 4, 64)
    for out, match in ((table.view(-1)[-2048:].view(BF).view(16, 4, 64), "out overlaps page_table"),
                       (on_lens, "out overlaps lengths"),
                       (q, "out overlaps q"), (both[0].view(-1)[:4096].view(16, 4, 64), "out overlaps the cache"),
                       (both[1].view(-1)[-6144:-2048].view(16, 4, 64), "out overlaps the cache"),
                       (both[1].view(-1)[-2048:].view(8, 4, 64), "GPU"), (fine, "GPU")):
        args = (q, kv, table, lens) if out.shape[0] == 16 else (q[:8], kv, table[:8], lens[:8])
        for given in (None, lse[:out.shape[0]]):
            with pytest.raises(ValueError, match=match):
                bd.bd_attend(*args, out=out, lse=given)
    for bad, match in ((table.view(torch.float32).view(-1)[:64].view(16, 4), "lse overlaps page_table"),
                       (lens.as_strided((64,), (1,)).view(torch.float32).view(16, 4), "lse overlaps lengths"),
                       (both[1].view(torch.float32).view(-1)[:64].view(16, 4), "lse overlaps the cache"),
                       (both[1].view(torch.float32).view(-1)[1024:1088].view(16, 4), "GPU")):
        for given in (None, fine):
            with pytest.raises(ValueError, match=match):
                bd.bd_attend(q, kv, table, lens, out=given, lse=bad)
    with pytest.raises(ValueError, match="lse overlaps out|out overlaps lse"):
        bd.bd_attend(q, kv, table, lens, out=fine, lse=fine.view(torch.float32).view(-1)[:64].view(16, 4))
    # scale bytes are read too
    s = [torch.zeros(16 * 4 * 64 * 2, dtype=torch.uint8) for _ in range(2)]
    k8, v8 = (torch.zeros((6, 2, 16, 64), dtype=torch.uint8).view(E4) for _ in range(2))
    kv = _cache(monkeypatch, k8, v8, *(t[:192].view(6, 2, 16) for t in s))
    for t in s:
        with pytest.raises(ValueError, match="out overlaps the cache"):
            bd.bd_attend(q, kv, table, lens, out=t.view(BF).view(16, 4, 64))


def test_the_ordinary_calls_outputs(monkeypatch):
    """What the short way takes for fine has to be: it is asked here about the cases above, on a device of its own."""
    from tenant_serving_amd import step
    both = [torch.zeros((6, 2, 2, 16, 64), dtype=BF) for _ in range(2)]
    kv = _cache(monkeypatch, both[0][:, 0], both[1][:, 0])
    q, out, lse = torch.zeros((16, 4, 64), dtype=BF), torch.zeros((16, 4, 64), dtype=BF), torch.zeros((16, 4))
    table, lens = torch.zeros((16, 2048), dtype=torch.int32), torch.zeros(16, dtype=torch.int32)
    q0 = q.data_ptr()

    def ask(out, lse=None):
        return step._attend_to(kv, q0, q0 + q.nbytes, table, lens, out, lse, 16, 4, -1)
    assert ask(out) and ask(out, lse) and ask(None, lse)
    assert not ask(q) and not ask(q, lse) and not ask(table.view(-1)[:2048].view(BF).view(16, 4, 64))
    assert not ask(both[0].view(-1)[:4096].view(16, 4, 64)) and not ask(out[:8]) and not ask(out.float())
    assert not ask(out, out.view(torch.float32).view(-1)[:64].view(16, 4))
    assert not ask(None, lens.view(torch.float32)[:, None].expand(16, 4))
    assert not ask(None, q.view(torch.float32).view(-1)[:64].view(16, 4))
    slots, rows = torch.zeros(16, dtype=torch.int32), [torch.zeros((16, 2, 64), dtype=BF) for _ in range(2)]

    def ask_read(out, slots=slots):
        return step._read_to(kv, out, slots, (16, 2, 64), -1)
    assert ask_read(rows) and ask_read(tuple(rows)) and not ask_read(rows[0]) and not ask_read([rows[0], rows[0]])
    assert not ask_read(rows, rows[1].view(torch.int32).view(-1)[:16]) and not ask_read([rows[0], rows[1].half()])
    assert not ask_read([rows[0], both[1].view(-1)[:2048].view(16, 2, 64)])


def test_addresses_against_rows_one_by_one():
    """The arithmetic behind the refusals, for random nested strides, against every byte of every row."""
    import random
    from tenant_serving_amd import step
    rng = random.Random(5)
    hits = 0
    for _ in range(300):
        row = rng.choice([1, 3, 8])
        extent, steps = row, []
        for _ in range(rng.randint(0, 3)):
            s, n = extent + rng.choice([0, 0, 1, 5]), rng.randint(2, 4)
            steps.insert(0, (s, n))
            extent = s * (n - 1) + extent
        base = 50
        starts = [base]
        for s, n in steps:
            starts = [a + i * s for a in starts for i in range(n)]
        held = {a + i for a in starts for i in range(row)}
        for _ in range(30):
            lo = rng.randint(30, base + extent + 10)
            size = rng.choice([0, 1, 2, 7, 40])
            want = bool(held & set(range(lo, lo + size)))
            hits += want
            assert step._on_rows(base, steps, row, lo, lo + size) == want
            if size:
                many = [rng.randint(30, base + extent + 10) for _ in range(rng.randint(1, 3))]
                want = any(held & set(range(a, a + size)) for a in many)
                assert step._any_on_rows(base, steps, row, torch.tensor(many), size) == want
    assert 1000 < hits < 8000
