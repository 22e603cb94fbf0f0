"""The 4-bit cache (e2m1 codes with a power-of-two scale per 32 columns): refusals on the host, and on the GPU what a
write holds, bit for bit, and what a read gives back, against tests/more_reference.py."""

import ctypes

import numpy as np
import pytest
import torch

import tenant_serving_amd as bd
from tenant_serving_amd import step
from tests import more_reference as ref

DEV = "cuda:0"
BF, F32, E2 = torch.bfloat16, torch.float32, torch.float4_e2m1fn_x2
FAKE = 1 << 20


def gen_of(seed):
    return torch.Generator().manual_seed(seed)


class Cache:
    """A 4-bit cache on the GPU, every byte of it random, and what it should hold, on the host."""

    def __init__(self, pages, heads, page, dim, layout="heads", seed=11, device=DEV):
        gen = gen_of(seed)
        self.heads, self.page, self.dim, self.slots = heads, page, dim, pages * page

        def fresh(*shape):
            return torch.randint(0, 256, shape, generator=gen, dtype=torch.uint8).to(device)
        row = dim // 2
        if layout == "both":
            base = fresh(pages, page, 2, heads, row).view(E2)
            k, v = (base[:, :, i].transpose(1, 2) for i in (0, 1))
        elif layout == "tokens":
            k, v = (fresh(pages, page, heads, row).view(E2).transpose(1, 2) for _ in range(2))
        else:
            k, v = (fresh(pages, heads, page, row).view(E2) for _ in range(2))
        scales = [fresh(pages, heads, dim // 32, page) for _ in range(2)]
        self.kv = bd.bd_kv_cache(k, v, *scales)
        self.rows = [t.cpu().view(torch.uint8).contiguous().numpy().copy() for t in (k, v)]
        self.scales = [t.cpu().numpy().copy() for t in scales]

    def expect(self, k, v, slots):
        for i, x in enumerate((k, v)):
            codes, bytes_ = ref.quantise4(x.double().numpy())
            packed = ref.pack4(codes)
            for t, s in enumerate(slots.tolist()):
                if 0 <= s < self.slots:
                    p, at = divmod(s, self.page)
                    self.rows[i][p, :, at], self.scales[i][p, :, :, at] = packed[t], bytes_[t]

    def check(self):
        for i, (t, s) in enumerate(((self.kv.k, self.kv.k_scales), (self.kv.v, self.kv.v_scales))):
            got = t.cpu().view(torch.uint8).contiguous().numpy()
            assert np.array_equal(s.cpu().numpy(), self.scales[i])
            off = got != self.rows[i]
            assert not off.any(), ("kv"[i], np.argwhere(off)[:4].tolist())

    def row64(self, which, slot):
        p, at = divmod(slot, self.page)
        return ref.decode4(ref.unpack4(self.rows[which][p, :, at]), self.scales[which][p, :, :, at])


def rows_of(T, heads, dim, dtype, seed):
    gen = gen_of(seed)
    x = torch.randn((T, heads, dim), generator=gen) * torch.exp2(torch.randint(-8, 9, (T, heads, 1), generator=gen).float())
    return x.to(dtype)


# ----------------------------------------------------------------------------
# on the host

def test_reference():
    """The plain form's own codes: every value of a group whose scale is known, and halfway ones."""
    x = np.zeros((1, 32))
    x[0, :16] = [6, 5, 5.001, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, 0.26, -6, -5, -0.25, -0.75, 0.0, 4]
    codes, byte = ref.quantise4(x)
    assert byte.tolist() == [[127]]
    assert codes[0, :16].tolist() == [7, 6, 7, 6, 4, 4, 2, 2, 0, 1, 15, 14, 8, 10, 0, 6]
    assert np.array_equal(ref.unpack4(ref.pack4(codes)), codes)
    # scale bytes by halving and doubling
    x = np.zeros((500, 32))
    x[:, 7] = np.random.default_rng(1).standard_normal(500).astype(np.float32) * 2.0 ** np.linspace(-140, 127, 500)
    x[:8, 7] = [6, 12, 3, 6 * 2.0 ** -125, 6.1 * 2.0 ** -125, 2.0 ** -149, 0, 1.5 * 2.0 ** 100]
    assert ref.quantise4(x)[1][:, 0].tolist() == [ref.scale_byte4(a) for a in np.abs(x).max(1)]
    assert ref.scale_byte4(0.0) == 2 and ref.scale_byte4(6.1) == 128 and ref.scale_byte4(3.0) == 126
    assert ref.scale_byte4(float(np.float32(3.4028234e38))) == 253


def test_c_refusals():
    lib = step._library()

    def kv(**change):
        d = dict(k=FAKE, v=FAKE, k_scales=FAKE, v_scales=FAKE, type=4, num_heads=2, head_dim=64, page_size=16,
                 num_pages=10, page_stride=1024, head_stride=512, token_stride=32)
        d.update(change)
        return step._KV(**d)
    pair = step._Pair
    for change, want in [(dict(k_scales=None), 1), (dict(v_scales=None), 1), (dict(head_dim=48), 2), (dict(head_dim=16), 2),
                         (dict(head_dim=288), 2), (dict(token_stride=24), 3), (dict(head_stride=520), 3),
                         (dict(page_stride=-16), 2), (dict(k_scales=FAKE + 4), 3), (dict(type=6), 5)]:
        d = kv(**change)
        r = ctypes.byref(d)
        assert lib.bd_kv_write(r, FAKE, pair(128, 64), FAKE, pair(128, 64), 0, FAKE, 4, None) == want, change
        assert lib.bd_kv_read(r, FAKE, 4, FAKE, FAKE, None) == want, change
    d = kv()
    assert lib.bd_kv_write(ctypes.byref(d), None, pair(128, 64), None, pair(128, 64), 0, None, 0, None) == 0
    assert lib.bd_kv_read(ctypes.byref(d), None, 0, None, None, None) == 0


def test_handle_refusals(monkeypatch):
    k, v = (torch.zeros((3, 2, 16, 32), dtype=torch.uint8).view(E2) for _ in range(2))
    s = [torch.zeros((3, 2, 2, 16), dtype=torch.uint8) for _ in range(2)]
    odd = torch.zeros((3, 2, 16, 24), dtype=torch.uint8).view(E2)
    for err, match, args in [(TypeError, "k must be", (k.view(torch.uint8), v, *s)), (TypeError, "k_scales", (k, v)),
                             (ValueError, "k_scales", (k, v, s[0][:, :, 0], s[1])),
                             (ValueError, "v_scales", (k, v, s[0], torch.zeros((3, 2, 16, 2), dtype=torch.uint8))),
                             (ValueError, "multiple of 32", (odd, odd.clone(), *s)),
                             (ValueError, "k and v", (k, v.view(torch.uint8), *s)),
                             (ValueError, "k_scales overlaps v_scales", (k, v, s[0], s[0])),
                             (ValueError, "k_scales overlaps k", (k, v, k.view(torch.uint8).view(-1)[:192].view(3, 2, 2, 16), s[1])),
                             (ValueError, "16 bytes", (torch.zeros((3, 2, 16, 40), dtype=torch.uint8).view(E2)[..., :32],
                                                       torch.zeros((3, 2, 16, 40), dtype=torch.uint8).view(E2)[..., :32], *s)),
                             (ValueError, "GPU", (k, v, *s))]:
        with pytest.raises(err, match=match):
            bd.bd_kv_cache(*args)
    with pytest.raises(ValueError, match="multiple of 32"):
        bd.bd_kv_cache.empty(3, 2, 16, 48, E2, "cpu")
    with monkeypatch.context() as m:
        m.setattr(step, "_same_gpu", lambda device, named: None)
        kv = bd.bd_kv_cache.empty(3, 2, 16, 64, E2, "cpu")
    kv._dev = 0
    assert kv.head_dim == 64 and kv.k.shape == (3, 2, 16, 32) and kv.k_scales.shape == (3, 2, 2, 16)
    rows, slots = torch.zeros((4, 2, 64), dtype=BF), torch.zeros(4, dtype=torch.int32)
    for args, match in (((torch.zeros((4, 2, 32), dtype=BF), rows, slots), "k must be"),
                        ((rows, rows.float(), slots), "one dtype"), ((rows, rows, slots[:3]), "slots"),
                        ((kv.k.view(BF).view(-1)[:512].view(4, 2, 64), rows, slots), "k overlaps the cache"),
                        ((rows, rows, kv.v_scales.view(torch.int32).view(-1)[:4]), "slots overlaps the cache")):
        with pytest.raises((ValueError, TypeError), match=match):
            bd.bd_kv_write(kv, *args)
    out = kv.k.view(BF).view(-1)[:512].view(4, 2, 64)
    with pytest.raises(ValueError, match=r"out\[0\] overlaps the cache"):
        bd.bd_kv_read(kv, slots, out=(out, rows))


# ----------------------------------------------------------------------------
# on the GPU

@pytest.mark.gpu
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("x_t", [BF, F32])
def test_write_and_read(dim, x_t):
    print("kv4", dim, x_t, flush=True)
    for heads, page, T, layout in ((1, 8, 1, "heads"), (3, 24, 61, "tokens"), (8, 16, 17, "both"), (2, 40, 130, "heads")):
        c = Cache(T // page + 4, heads, page, dim, layout)
        slots = torch.randperm(c.slots, generator=gen_of(T))[:T].to(torch.int32)
        k, v = rows_of(T, heads, dim, x_t, 1), rows_of(T, heads, dim, x_t, 2)
        c.expect(k, v, slots)
        bd.bd_kv_write(c.kv, k.to(DEV), v.to(DEV), slots.to(DEV))
        c.check()
        for i, r in enumerate(bd.bd_kv_read(c.kv, slots.to(DEV))):
            assert r.dtype == BF and r.shape == (T, heads, dim)
            assert np.array_equal(r.cpu().double().numpy(), np.stack([c.row64(i, s) for s in slots.tolist()]))


@pytest.mark.gpu
def test_values():
    """Ties, borders of the scale, signed zeros, subnormals, the largest numbers, NaN and infinities."""
    mid = (ref.E2M1[1:] + ref.E2M1[:-1]) / 2
    ties = torch.from_numpy(np.resize(np.concatenate([[6.0], mid, -mid]), 32)).float().view(1, 32)
    rows = [ties, ties * 2.0 ** -20, ties * 2.0 ** 100, ties * 2.0 ** -127, ties * 2.0 ** -140, torch.zeros(1, 32), -torch.zeros(1, 32),
            torch.full((1, 32), 2.0 ** -149), torch.full((1, 32), 3.4028234e38), torch.linspace(0, 6, 32)[None],
            torch.linspace(0, 6.0001, 32)[None], torch.linspace(-3, 3.0001, 32)[None], torch.linspace(1e-38, 1e-37, 32)[None],
            torch.full((1, 32), float("nan")), torch.full((1, 32), -float("inf"))]
    mixed = torch.randn((4, 32), generator=gen_of(8))
    mixed[0, 5], mixed[1, 6], mixed[2, 31] = float("nan"), float("inf"), -float("inf")
    rows = torch.cat(rows + [mixed])
    n = rows.shape[0]
    for x_t in (F32, BF):
        both = torch.stack((rows, rows.flip(0)), 1).view(n, 1, 64).to(x_t)      # a good group next to a bad one
        c = Cache(5, 1, 8, 64)
        v = both.flip(0).contiguous()
        slots = torch.arange(n, dtype=torch.int32)
        c.expect(both, v, slots)
        bd.bd_kv_write(c.kv, both.to(DEV), v.to(DEV), slots.to(DEV))
        c.check()
        for i, r in enumerate(bd.bd_kv_read(c.kv, slots.to(DEV))):
            want = np.stack([c.row64(i, s) for s in range(n)])
            want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)   # past bf16's range
            assert np.array_equal(r.cpu().double().numpy(), want, equal_nan=True)


@pytest.mark.gpu
def test_any_byte_reads_as_defined():
    """All 256 scale bytes with all codes, as they may lie in a cache."""
    c = Cache(16, 1, 16, 32)
    codes = torch.arange(256 * 16).to(torch.uint8).view(16, 1, 16, 16)
    c.kv.k.view(torch.uint8).copy_(codes.to(DEV))
    c.kv.k_scales.copy_(torch.arange(256).to(torch.uint8).view(16, 1, 1, 16).to(DEV))
    slots = torch.arange(256, dtype=torch.int32)
    got = bd.bd_kv_read(c.kv, slots.to(DEV))[0].cpu().double().numpy()[:, 0]
    want = ref.decode4(ref.unpack4(codes.numpy().reshape(256, 16)), np.arange(256).reshape(256, 1))
    want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)
    assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.gpu
def test_strided_inputs_and_slots():
    """Views of one q, k, v result; slots out of range and named twice, in short calls and long ones."""
    T, heads, dim = 37, 4, 96
    for x_t in (F32, BF):
        qkv = torch.randn((T, 6 * heads * dim + 16), generator=gen_of(3)).to(x_t)
        k = qkv[:, 2 * heads * dim:3 * heads * dim].view(T, heads, dim)
        v = qkv[:, 5 * heads * dim:6 * heads * dim].view(T, heads, dim)
        c = Cache(7, heads, 8, dim, "both")
        slots = torch.randint(-3, c.slots + 3, (T,), generator=gen_of(4)).to(torch.int32)
        slots[0] = slots[T - 1] = 7
        slots[1], slots[2] = -2 ** 31, 2 ** 31 - 1
        c.expect(k, v, slots)
        g = qkv.to(DEV)
        bd.bd_kv_write(c.kv, g[:, 2 * heads * dim:3 * heads * dim].view(T, heads, dim),
                       g[:, 5 * heads * dim:6 * heads * dim].view(T, heads, dim), slots.to(DEV))
        c.check()
    for T in (700, 5000, 33000):
        c = Cache(T // 24 + 3, 1, 16, 32)
        slots = torch.randint(-3, c.slots + 3, (T,), generator=gen_of(T)).to(torch.int32)
        k, v = rows_of(T, 1, 32, BF, 5), rows_of(T, 1, 32, BF, 6)
        c.expect(k, v, slots)
        bd.bd_kv_write(c.kv, k.to(DEV), v.to(DEV), slots.to(DEV))
        c.check()
    r = bd.bd_kv_read(c.kv, torch.tensor([-1, c.slots, 0], dtype=torch.int32, device=DEV))[0]
    assert (r[0] == 0).all() and r[1].isnan().all() and r[2].isfinite().all()


@pytest.mark.gpu
def test_rows_past_32_bits():
    """Codes and scale bytes at the far end of arrays of more than 4 GiB."""
    heads, page, dim = 8, 16, 128
    pages = (1 << 32) // (heads * page * dim // 2) + 40
    kv = bd.bd_kv_cache.empty(pages, heads, page, dim, E2, DEV)
    slots = torch.tensor([pages * page - 1, 0, pages * page // 2 + 3, pages * page - 700], dtype=torch.int32)
    k, v = rows_of(4, heads, dim, BF, 1), rows_of(4, heads, dim, BF, 2)
    bd.bd_kv_write(kv, k.to(DEV), v.to(DEV), slots.to(DEV))
    for x, got in zip((k, v), bd.bd_kv_read(kv, slots.to(DEV))):
        codes, bytes_ = ref.quantise4(x.double().numpy())
        assert np.array_equal(got.cpu().double().numpy(), ref.decode4(codes, bytes_))
    assert int(kv.k_scales[pages - 1, 3, 2, 15]) == int(ref.quantise4(k[0].double().numpy())[1][3, 2])
