"""GPU parity of the step operators (include/bitdelta_step.h) against the plain 64-bit implementations of
tests/step_reference.py on the same seeded inputs.

Tolerances, from the roundings the calls document (u = 2^-24, half a step of fp32):
- bf16 results: half a step is 2^-8 of the value;
- e4m3 results: half a step is 2^-4 of the value, or 2^-10 of the scale among subnormal codes;
- norm: fp32 sum of d squares, root, division, two products: (d / 2 + 16) u of the value;
- attention, with S the largest sum of |q k| scale over a row: a score is off by at most ds = (D + 8) u S, plus
  2^-15 S for fp32 queries (two bf16 terms leave 2^-16 of each factor); a weight by a factor exp(2 ds) (its own score
  and the maximum's) and 2^-15 for its two bf16 terms and the exponential; sums add (n + 64) u of the largest value.
"""

import numpy as np
import pytest
import torch

from tests import step_reference as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def bd():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tenant_serving_amd as m
    m.library()  # raises if the HIP library is missing: no silent fallback
    return m


def gen_of(seed):
    return torch.Generator().manual_seed(seed)


def same_bits(a, b):
    a, b = a.detach().cpu().contiguous(), b.detach().cpu().contiguous()
    return a.dtype == b.dtype and a.shape == b.shape and torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ----------------------------------------------------------------------------
# norm

def norm_inputs(M, d, x_t, res_t, g_t, V, seed=5):
    gen = gen_of(seed + 17 * M + d)
    x = torch.randn((M, d), generator=gen).mul(3).to(x_t)
    res = None if res_t is None else torch.randn((M, d), generator=gen).mul(20).to(res_t)
    gain = (1 + 0.3 * torch.randn((V, d), generator=gen)).to(g_t)
    ids = torch.randint(0, V, (M,), generator=gen, dtype=torch.int32)
    return x, res, gain, ids


def on_gpu(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def check_bf16(got, want, d):
    got = ref.to64(got)
    tol = np.abs(want) * (2.0 ** -8 + (d / 2 + 16) * U) + 2.0 ** -133
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    assert np.all((np.abs(got - want) <= tol)[~nan])


def check_e4m3(codes, scales, want, d):
    codes, scales = codes.cpu().view(torch.uint8).numpy(), scales.cpu().numpy()
    assert scales.shape == (want.shape[0], (d + 31) // 32)
    for g in range(scales.shape[1]):
        part = want[:, 32 * g:32 * g + 32]
        for r in range(part.shape[0]):
            byte = int(scales[r, g])
            if np.isnan(part[r]).any():
                assert np.all(codes[r, 32 * g:32 * g + 32] & 127 == 127)
                continue
            amax, off = np.abs(part[r]).max(), (d / 2 + 16) * U
            assert ref.scale_byte(amax * (1 - off)) <= byte <= ref.scale_byte(amax * (1 + off))
            got = ref.decode(codes[r, 32 * g:32 * g + 32], byte)
            tol = np.maximum(np.abs(part[r]) * 2.0 ** -4, 2.0 ** -10 * 2.0 ** (byte - 127)) + np.abs(part[r]) * off
            assert np.all(np.abs(got - part[r]) <= tol)


@pytest.mark.parametrize("M,d", [(1, 8), (3, 40), (5, 512), (2, 520), (7, 2048), (4, 2056), (3, 4096), (2, 4104),
                                 (9, 8192), (3, 8200), (2, 16384), (1, 16392), (2, 32768), (1, 32776), (1, 65536)])
@pytest.mark.parametrize("x_t,res_t", [(BF, None), (F32, BF), (BF, F32), (F32, F32), (BF, BF), (F32, None)])
def test_norm(bd, M, d, x_t, res_t):
    print("norm", M, d, x_t, res_t, flush=True)
    for g_t, V in ((BF, 3), (F32, 1)):
        x, res, gain, ids = norm_inputs(M, d, x_t, res_t, g_t, V)
        want, res_want = ref.rms_norm(x, gain, 1e-5, res, ids)
        gx, gr, gg, gi = on_gpu(x, res, gain, ids)
        keep = None if gr is None else gr.clone()
        y = bd.bd_rms_norm(gx, gg, 1e-5, residual=gr, variant_ids=gi)
        c = bd.bd_rms_norm_e4m3(gx, gg, 1e-5, residual=gr, variant_ids=gi)
        if res is not None:
            assert same_bits(y[1], res_want) and same_bits(c[2], res_want) and same_bits(gr, keep)
            y = y[0]
        assert y.dtype == BF and c[0].dtype == E4
        check_bf16(y, want, d)
        check_e4m3(c[0], c[1], want, d)


@pytest.mark.parametrize("d", [6144, 6152, 12288, 12296, 16376, 24576, 24584])
def test_norm_between_widths(bd, d):
    test_norm(bd, 2, d, F32, BF)
    test_norm(bd, 2, d, BF, F32)
    test_norm(bd, 2, d, BF, None)


def test_norm_products_below_fp32(bd):
    """Products between 0 and the least fp32 number, whose codes are zeros, next to larger ones."""
    d = 96
    x = torch.full((3, d), 2.0 ** -30)
    x[:, ::3] *= -1
    x[:, 5] = 1.0
    x[2, 40] = float("nan")
    gain = torch.full((d,), 2.0 ** -133).to(BF)
    gain[::7] *= -1
    gain[5], gain[70] = 2.0 ** -100, 0.0
    codes, scales = bd.bd_rms_norm_e4m3(x.to(DEV), gain.to(DEV), 1e-5)
    want, _ = ref.rms_norm(x, gain[None], 1e-5)
    assert 0 < np.abs(want[0, 6]) < 2.0 ** -150
    check_e4m3(codes, scales, want, d)
    assert ((codes[:2].cpu().view(torch.uint8)[:, 6:] & 127) == 0).all()


def test_norm_forms(bd):
    x, res, gain, ids = on_gpu(*norm_inputs(6, 72, F32, BF, BF, 4))
    y, r = bd.bd_rms_norm(x, gain, residual=res, variant_ids=ids)
    # leading dimensions, given outputs, in place, a single gain
    y2, r2 = bd.bd_rms_norm(x.view(2, 3, 72), gain, residual=res.view(2, 3, 72), variant_ids=ids.view(2, 3))
    assert same_bits(y2.view(6, 72), y) and same_bits(r2.view(6, 72), r)
    out, ro = torch.empty_like(y), torch.empty_like(r)
    a, b = bd.bd_rms_norm(x, gain, residual=res, variant_ids=ids, residual_out=ro, out=out)
    assert a is out and b is ro and same_bits(out, y) and same_bits(ro, r)
    c, s, r3 = bd.bd_rms_norm_e4m3(x, gain, residual=res, variant_ids=ids)
    cc, ss = torch.empty_like(c), torch.empty_like(s)
    bd.bd_rms_norm_e4m3(x, gain, residual=res, variant_ids=ids, out=cc, scales=ss)
    assert same_bits(c, cc) and same_bits(s, ss) and same_bits(r3, r)
    inplace = res.clone()
    y3, r4 = bd.bd_rms_norm(x, gain, residual=inplace, variant_ids=ids, residual_out=inplace)
    assert r4 is inplace and same_bits(inplace, r) and same_bits(y3, y)
    one = bd.bd_rms_norm(x, gain[2])
    assert same_bits(one, bd.bd_rms_norm(x, gain, variant_ids=torch.full_like(ids, 2)))
    assert same_bits(bd.bd_rms_norm(x, gain), bd.bd_rms_norm(x, gain[0]))
    assert bd.bd_rms_norm(x[:0], gain).shape == (0, 72)
    for bad in (dict(out=x.view(torch.bfloat16).view(-1)[:6 * 72].view(6, 72)), dict(residual=res, out=res),
                dict(residual=res, residual_out=y, out=y)):
        with pytest.raises(ValueError, match="overlaps"):
            bd.bd_rms_norm(x, gain, **bad)
    with pytest.raises(ValueError, match="expected"):
        bd.bd_rms_norm(x, gain.cpu())


@pytest.mark.parametrize("d", [64, 520, 8192, 8200])
def test_norm_ids_and_specials(bd, d):
    """Ids out of range give NaN rows; NaN and infinities stay in their row; zeros give zeros (of the gain's sign)."""
    x, res, gain, _ = norm_inputs(8, d, F32, BF, BF, 3)
    ids = torch.tensor([0, -1, 3, 2 ** 31 - 1, -2 ** 31, 1, 2, 0], dtype=torch.int32)
    x[5, d // 2] = float("nan")
    x[6, 3] = float("inf")
    x[7] = 0
    res[7] = 0
    want, res_want = ref.rms_norm(x, gain, 1e-5, res, ids)
    with np.errstate(all="ignore"):
        assert np.isnan(want[[1, 2, 3, 4, 5]]).all() and np.isnan(want[6, 3]) and not np.isnan(want[6, 4])
    gx, gr, gg, gi = on_gpu(x, res, gain, ids)
    y, r = bd.bd_rms_norm(gx, gg, residual=gr, variant_ids=gi)
    assert torch.equal(r.cpu().nan_to_num(7.5), res_want.nan_to_num(7.5))
    check_bf16(y, want, d)
    codes, scales, _ = bd.bd_rms_norm_e4m3(gx, gg, residual=gr, variant_ids=gi)
    cu = codes.cpu().view(torch.uint8)
    assert ((cu[1:6] & 127) == 127).all() and (scales.cpu()[1:5] == 127).all()
    assert (cu[6, 3] & 127) == 127 and ((cu[6, torch.arange(d) != 3] & 127) == 0).all()
    assert ((cu[7] & 127) == 0).all() and (scales.cpu()[7] == 16).all()
    check_e4m3(codes[:1], scales[:1], want[:1], d)


def test_norm_many_rows(bd):
    x, _, gain, _ = norm_inputs(1, 8, BF, None, BF, 1)
    M = (1 << 21) + 77          # more rows than one launch takes
    g = torch.randn((M, 8), generator=torch.Generator(device=DEV).manual_seed(3), device=DEV).to(BF)
    y = bd.bd_rms_norm(g, gain.to(DEV))
    for at in (0, (1 << 21) - 1, 1 << 21, M - 1):
        want, _ = ref.rms_norm(g[at:at + 1], gain, 1e-5)
        check_bf16(y[at:at + 1], want, 8)


@pytest.mark.parametrize("x_t,d", [(BF, 28672), (F32, 8192), (BF, 512), (BF, 2056)])
def test_norm_large(bd, x_t, d):
    """Inputs beyond the last-level cache, which are loaded another way, against the same rows in a small call."""
    M = (200 << 20) // (d * (6 if x_t == F32 else 4)) + 3
    g = torch.Generator(device=DEV).manual_seed(d)
    x = torch.randn((M, d), generator=g, device=DEV, dtype=x_t)
    res = torch.randn((M, d), generator=g, device=DEV, dtype=BF)
    gain = torch.randn((2, d), generator=g, device=DEV).to(BF)
    ids = torch.arange(M, device=DEV, dtype=torch.int32) % 2
    y, r = bd.bd_rms_norm(x, gain, residual=res, variant_ids=ids)
    c, s, r2 = bd.bd_rms_norm_e4m3(x, gain, residual=res, variant_ids=ids)
    for a in (0, M // 2, M - 16):
        part = slice(a, a + 16)
        y2, r3 = bd.bd_rms_norm(x[part], gain, residual=res[part], variant_ids=ids[part])
        c2, s2, _ = bd.bd_rms_norm_e4m3(x[part], gain, residual=res[part], variant_ids=ids[part])
        assert same_bits(y[part], y2) and same_bits(r[part], r3) and same_bits(r2[part], r3)
        assert same_bits(c[part], c2) and same_bits(s[part], s2)


# ----------------------------------------------------------------------------
# the cache

class Cache:
    """A cache on the GPU and what it should hold, on the host."""

    def __init__(self, bd, pages, heads, page, dim, kind, layout="heads", seed=11):
        gen = gen_of(seed)
        self.kind, self.heads, self.page, self.dim = kind, heads, page, dim
        shape = (pages, heads, page, dim) if layout == "heads" else (pages, page, heads, dim)
        if layout == "both":
            shape = (pages, page, 2, heads, dim)
        self.bytes = 1 if kind == E4 else 2

        def fresh():
            return torch.randint(0, 256, (*shape[:-1], dim * self.bytes), generator=gen, dtype=torch.uint8)
        if layout == "both":
            base = fresh().to(DEV).view(kind)
            k, v = (base[:, :, i].transpose(1, 2) for i in (0, 1))
        else:
            k, v = (fresh().to(DEV).view(kind) for _ in range(2))
            if layout == "tokens":
                k, v = k.transpose(1, 2), v.transpose(1, 2)
        ks = vs = None
        if kind == E4:
            ks, vs = (torch.randint(0, 256, (pages, heads, page), generator=gen, dtype=torch.uint8).to(DEV)
                      for _ in range(2))
        self.kv = bd.bd_kv_cache(k, v, ks, vs)
        self.rows = [t.cpu().contiguous().view(torch.uint8).numpy().reshape(pages, heads, page, dim * self.bytes).copy()
                     for t in (k, v)]
        self.scales = None if ks is None else [t.cpu().numpy().copy() for t in (ks, vs)]
        self.slots = pages * page

    def expect(self, k, v, slots):
        for t, s in enumerate(slots.tolist()):
            if not 0 <= s < self.slots:
                continue
            p, at = divmod(s, self.page)
            for i, x in enumerate((k, v)):
                if self.kind == E4:
                    codes, byte = ref.quantise(ref.to64(x[t]))
                    self.rows[i][p, :, at], self.scales[i][p, :, at] = codes, byte
                else:
                    self.rows[i][p, :, at] = x[t].to(BF).contiguous().view(torch.uint8).numpy()

    def check(self):
        for i, t in enumerate((self.kv.k, self.kv.v)):
            got = t.cpu().contiguous().view(torch.uint8).numpy().reshape(self.rows[i].shape)
            if self.kind == E4:
                # any NaN code will do for NaN
                a, b = got & 127, self.rows[i] & 127
                off = np.where(b == 127, a != 127, got != self.rows[i])
            else:
                a, b = got.view(np.uint16), self.rows[i].view(np.uint16)
                off = np.where((b & 0x7fff) > 0x7f80, (a & 0x7fff) <= 0x7f80, a != b)
            assert not off.any(), ("kv"[i], np.argwhere(off)[:4].tolist())
        if self.scales:
            assert np.array_equal(self.kv.k_scales.cpu().numpy(), self.scales[0])
            assert np.array_equal(self.kv.v_scales.cpu().numpy(), self.scales[1])

    def row64(self, which, slot):
        p, at = divmod(slot, self.page)
        r = self.rows[which][p, :, at]
        if self.kind == E4:
            return np.stack([ref.decode(r[h], self.scales[which][p, h, at]) for h in range(self.heads)])
        return torch.from_numpy(r.copy()).view(BF).double().numpy()


def rows_of(T, heads, dim, dtype, seed):
    gen = gen_of(seed)
    x = torch.randn((T, heads, dim), generator=gen) * torch.exp2(torch.randint(-8, 9, (T, heads, 1), generator=gen).float())
    return x.to(dtype)


@pytest.mark.parametrize("dim", [16, 64, 80, 128, 144, 208, 256])
@pytest.mark.parametrize("kind", [BF, E4])
@pytest.mark.parametrize("x_t", [BF, F32])
def test_kv_write_and_read(bd, dim, kind, x_t):
    print("kv", dim, kind, x_t, flush=True)
    for heads, page, T, layout in ((1, 8, 1, "heads"), (3, 24, 61, "tokens"), (8, 16, 17, "both"), (2, 40, 130, "heads")):
        c = Cache(bd, T // page + 4, heads, page, dim, kind, layout)
        slots = torch.randperm(c.slots, generator=gen_of(T))[:T].to(torch.int32)
        k, v = rows_of(T, heads, dim, x_t, 1), rows_of(T, heads, dim, x_t, 2)
        c.expect(k, v, slots)
        bd.bd_kv_write(c.kv, k.to(DEV), v.to(DEV), slots.to(DEV))
        c.check()
        rk, rv = bd.bd_kv_read(c.kv, slots.to(DEV))
        for i, r in enumerate((rk, rv)):
            assert r.dtype == BF and r.shape == (T, heads, dim)
            assert np.array_equal(ref.to64(r), np.stack([c.row64(i, s) for s in slots.tolist()]))


def test_kv_write_strided_inputs(bd):
    T, heads, dim = 37, 4, 64
    for x_t, kind in ((F32, E4), (BF, BF), (F32, BF), (BF, E4)):
        qkv = torch.randn((T, 6 * heads * dim + 16), generator=gen_of(3)).to(x_t)
        k = qkv[:, 2 * heads * dim:3 * heads * dim].view(T, heads, dim)
        v = rows_of(heads, T, dim, x_t, 9).transpose(0, 1)      # heads outermost
        c = Cache(bd, 7, heads, 8, dim, kind)
        slots = torch.randperm(c.slots, generator=gen_of(4))[:T].to(torch.int32)
        c.expect(k, v, slots)
        g = qkv.to(DEV)
        gv = v.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)
        bd.bd_kv_write(c.kv, g[:, 2 * heads * dim:3 * heads * dim].view(T, heads, dim), gv, slots.to(DEV))
        c.check()


def test_kv_slots_out_of_range_and_named_twice(bd):
    """Skipped slots leave the cache as it was; of several tokens with one slot the last stays, wherever they are."""
    for kind in (BF, E4):
        for T in (5, 64, 700, 5000):
            c = Cache(bd, 40, 1, 16, 16, kind)
            gen = gen_of(T)
            slots = torch.randint(-3, c.slots + 3, (T,), generator=gen).to(torch.int32)
            slots[0] = slots[T - 1] = 7
            slots[1], slots[2] = -2 ** 31, 2 ** 31 - 1
            k, v = rows_of(T, 1, 16, BF, 5), rows_of(T, 1, 16, BF, 6)
            c.expect(k, v, slots)
            for _ in range(2):
                bd.bd_kv_write(c.kv, k.to(DEV), v.to(DEV), slots.to(DEV))
                c.check()
    for kind in (BF, E4):
        c = Cache(bd, 3, 2, 8, 32, kind)
        slots = torch.tensor([-1, 23, 24, 2 ** 31 - 1, -2 ** 31, 0], dtype=torch.int32)
        rk, rv = bd.bd_kv_read(c.kv, slots.to(DEV))
        for r in (rk, rv):
            assert (r[0] == 0).all() and (r[4] == 0).all() and r[2].isnan().all() and r[3].isnan().all()
        out = torch.empty((6, 2, 32), dtype=BF, device=DEV), torch.empty((6, 2, 32), dtype=BF, device=DEV)
        got = bd.bd_kv_read(c.kv, slots.to(DEV), out=out)
        assert got[0] is out[0] and same_bits(out[0], rk) and same_bits(out[1], rv)
        none = torch.empty(0, dtype=torch.int32, device=DEV)
        assert bd.bd_kv_read(c.kv, none)[0].shape == (0, 2, 32)
        bd.bd_kv_write(c.kv, out[0][:0], out[1][:0], none)
        c.check()


@pytest.mark.parametrize("T,start", [(4096, 1), (4097, 2), (9001, 3), (70001, 1), (300001, 0)])
def test_kv_write_many_with_repeats(bd, T, start):
    """Long calls with many slots named again, near and far, from slot arrays at any 4-byte border."""
    page, pages = 16, T // 24 + 3
    kv = bd.bd_kv_cache.empty(pages, 1, page, 16, BF, DEV)
    kv.k.zero_(), kv.v.zero_()
    gen = gen_of(T)
    slots = torch.randint(-2, pages * page + 2, (T + start,), generator=gen).to(torch.int32)
    slots[start + 5:start + 40] = slots[start + 3]
    k = torch.arange(T).float().view(T, 1, 1).expand(T, 1, 16)
    # token numbers in two exact bf16 parts
    hi, lo = (torch.div(k, 256, rounding_mode="floor") * 1.0).to(BF), (k % 256).to(BF)
    bd.bd_kv_write(kv, hi.contiguous().to(DEV), lo.contiguous().to(DEV), slots.to(DEV)[start:])
    want = np.full(pages * page, -1, np.int64)
    own = slots[start:].numpy()
    ok = (own >= 0) & (own < pages * page)
    want[own[ok]] = np.arange(T)[ok]          # the last assignment stays
    got_hi = kv.k.float().cpu().numpy()[:, 0].reshape(-1, 16)
    got_lo = kv.v.float().cpu().numpy()[:, 0].reshape(-1, 16)
    w_hi = torch.from_numpy(np.where(want < 0, 0, want // 256)).float().to(BF).float().numpy()
    w_lo = np.where(want < 0, 0, want % 256)
    assert (got_hi == w_hi[:, None]).all() and (got_lo == w_lo[:, None]).all()


def test_kv_values(bd):
    """Ties, borders of the scale, signed zeros, subnormals, the largest numbers, NaN and infinities."""
    dim = 32
    ties = torch.from_numpy(np.resize((ref.E4M3[1:] + ref.E4M3[:-1]) / 2, 4 * dim)).float().view(4, dim)
    ties[:, 0] = 448
    rows = torch.cat([
        ties, -ties * 2.0 ** -30, torch.zeros(1, dim), -torch.zeros(1, dim), torch.full((1, dim), 2.0 ** -149),
        torch.full((1, dim), 3.4028234e38), torch.linspace(0, 448, dim)[None], torch.linspace(0, 449, dim)[None],
        torch.linspace(1e-36, 1e-34, dim)[None], torch.full((1, dim), float("nan")), torch.full((1, dim), -float("inf"))])
    mixed = torch.randn((3, dim), generator=gen_of(8))
    mixed[0, 5], mixed[1, 6], mixed[2, 7] = float("nan"), float("inf"), -float("inf")
    rows = torch.cat([rows, mixed])
    T = rows.shape[0]
    for kind in (E4, BF):
        for x_t in (F32, BF):
            c = Cache(bd, 5, 1, 8, dim, kind)
            k = rows.to(x_t).view(T, 1, dim)
            v = k.flip(0).contiguous()
            slots = torch.arange(T, dtype=torch.int32)
            c.expect(k, v, slots)
            bd.bd_kv_write(c.kv, k.to(DEV), v.to(DEV), slots.to(DEV))
            c.check()
            r = ref.to64(bd.bd_kv_read(c.kv, slots.to(DEV))[0])
            want = np.stack([c.row64(0, s) for s in range(T)])
            # the largest fp32 rounds up to the e4m3 value 2^128, which is infinity in bf16 (whose own rounding of it
            # gives infinity as well)
            want = np.where(np.abs(want) == 2.0 ** 128, np.copysign(np.inf, want), want)
            off = np.where(np.isnan(want), ~np.isnan(r), r != want)
            assert not off.any(), [(int(a), r[a, 0, e], want[a, 0, e]) for a, _, e in np.argwhere(off)[:6]]


# ----------------------------------------------------------------------------
# attention

def attend_case(bd, lens, heads, group, dim, page, kind, q_t, layout="heads", seed=21, spread=1.0, spare=3):
    gen = gen_of(seed)
    B, most = len(lens), max(1, max(-(-n // page) for n in lens))
    need = sum(-(-n // page) for n in lens) + spare
    c = Cache(bd, need, heads, page, dim, kind, layout, seed)      # random bytes behind every last token: NaN too
    order = torch.randperm(need, generator=gen).tolist()
    table = torch.full((B, most), -1, dtype=torch.int32)
    slots = []
    for b, n in enumerate(lens):
        for i in range(-(-n // page)):
            table[b, i] = order.pop()
        slots += [int(table[b, t // page]) * page + t % page for t in range(n)]
    T = len(slots)
    slots = torch.tensor(slots, dtype=torch.int32)
    k = (torch.randn((T, heads, dim), generator=gen) * spread).to(BF)
    v = torch.randn((T, heads, dim), generator=gen).to(BF)
    q = (torch.randn((B, heads * group, dim), generator=gen) * 2).to(q_t)
    if T:
        c.expect(k, v, slots)
        bd.bd_kv_write(c.kv, k.to(DEV), v.to(DEV), slots.to(DEV))
    return c, q, table, torch.tensor(lens, dtype=torch.int32), slots.tolist()


def check_attend(c, q, lens, slots, out, lse, scale, rows=None):
    B, hq, dim = q.shape
    out, lse, q64 = ref.to64(out), ref.to64(lse), ref.to64(q)
    at = 0
    for b, n in enumerate(lens):
        own = slots[at:at + n]
        at += n
        if rows is not None and b not in rows:
            continue
        kr = np.stack([c.row64(0, s) for s in own]) if n else np.zeros((0, c.heads, dim))
        vr = np.stack([c.row64(1, s) for s in own]) if n else np.zeros((0, c.heads, dim))
        want, want_lse, S = ref.attend(q64[b], kr, vr, scale)
        ds = (dim + 8) * U * S + (2.0 ** -15 * S if q.dtype == F32 else 0.0)
        fine = np.abs(vr[np.isfinite(vr)])
        vmax = fine.max() if fine.size else 0.0
        tol = 2.0 ** -8 * np.abs(want) + 2 * vmax * (np.expm1(2 * ds) + 2.0 ** -15 + (n + 64) * U) + 2.0 ** -133
        assert np.array_equal(np.isnan(out[b]), np.isnan(want)), b
        ok = ~np.isnan(want)
        assert np.all(np.abs(out[b] - want)[ok] <= tol[ok]), (b, n, np.abs(out[b] - want)[ok].max())
        okl = np.isfinite(want_lse)
        assert np.array_equal(lse[b][~okl], want_lse[~okl], equal_nan=True)
        tl = ds + (n + 64) * U + 4 * U * np.abs(want_lse[okl])
        assert np.all(np.abs(lse[b][okl] - want_lse[okl]) <= tl), (b, n)


def run_attend(bd, c, q, table, lens, scale=None):
    lse = torch.empty(q.shape[:2], dtype=F32, device=DEV)
    out = bd.bd_attend(q.to(DEV), c.kv, table.to(DEV), lens.to(DEV), scale, lse=lse)
    return out, lse


EDGES = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 160, 255, 256, 257, 300]


@pytest.mark.parametrize("dim", [16, 64, 80, 128, 144, 256])
@pytest.mark.parametrize("kind", [BF, E4])
@pytest.mark.parametrize("q_t", [BF, F32])
def test_attend_lengths(bd, dim, kind, q_t):
    print("attend", dim, kind, q_t, flush=True)
    for heads, group, page, layout in ((2, 4, 16, "heads"), (1, 8, 24, "tokens")):
        c, q, table, lens, slots = attend_case(bd, EDGES, heads, group, dim, page, kind, q_t, layout)
        out, lse = run_attend(bd, c, q, table, lens)
        assert out.dtype == BF and out.shape == q.shape
        check_attend(c, q, EDGES, slots, out, lse, dim ** -0.5)


@pytest.mark.parametrize("heads,group", [(1, 1), (3, 1), (2, 2), (1, 7), (2, 16), (1, 17), (2, 33), (1, 64), (9, 3)])
def test_attend_head_layouts(bd, heads, group):
    print("attend heads", heads, group, flush=True)
    for kind, dim, page in ((E4, 64, 8), (BF, 128, 48)):
        lens = [5, 0, 131, 64, 200]
        c, q, table, lens_t, slots = attend_case(bd, lens, heads, group, dim, page, kind, BF, "both")
        out, lse = run_attend(bd, c, q, table, lens_t)
        check_attend(c, q, lens, slots, out, lse, dim ** -0.5)


@pytest.mark.parametrize("lens", [[5000], [1, 3000, 2], [129] * 40, [0] * 7 + [2049], [700, 0, 1500, 1, 64, 2000],
                                  [3] * 130, list(range(70))])
@pytest.mark.parametrize("kind", [BF, E4])
def test_attend_splits(bd, lens, kind):
    """Rows that many workgroups share, rows that share a workgroup, more sequences than a wave has lanes."""
    print("attend split", lens[:6], len(lens), kind, flush=True)
    c, q, table, lens_t, slots = attend_case(bd, lens, 2, 3, 32, 16, kind, F32)
    out, lse = run_attend(bd, c, q, table, lens_t)
    check_attend(c, q, lens, slots, out, lse, 32 ** -0.5)
    again, lse2 = run_attend(bd, c, q, table, lens_t)
    assert same_bits(out, again) and same_bits(lse, lse2)


def test_attend_every_workgroup(bd):
    """More units than workgroups: every one of them has several, rows start and end inside them."""
    lens = [(97 * i) % 1400 for i in range(48)]
    c, q, table, lens_t, slots = attend_case(bd, lens, 4, 2, 16, 8, BF, BF)
    out, lse = run_attend(bd, c, q, table, lens_t)
    check_attend(c, q, lens, slots, out, lse, 0.25)


@pytest.mark.parametrize("heads,dim,kind", [(8, 16, BF), (4, 64, E4), (2, 128, BF), (3, 208, E4)])
def test_attend_more_rows_than_workgroups(bd, heads, dim, kind):
    """More (sequence, head) rows than workgroups, short ones among long ones, so that rows of every length are cut."""
    B = 800 // heads
    lens = [(37 * i) % 150 for i in range(B)]
    for i, n in ((3, 2000), (B // 2, 1300), (B - 2, 777)):
        lens[i] = n
    c, q, table, lens_t, slots = attend_case(bd, lens, heads, 2, dim, 16, kind, BF)
    out, lse = run_attend(bd, c, q, table, lens_t)
    check_attend(c, q, lens, slots, out, lse, dim ** -0.5,
                 rows=(0, 1, 2, 3, 4, 5, B // 2 - 1, B // 2, B // 2 + 1, B - 3, B - 2, B - 1))


def test_attend_many_sequences(bd):
    """Thousands of sequences that share their pages: rows of the batch are what they are alone."""
    lens = [0, 1, 30, 64, 130, 7, 128, 129]
    c, q, table, lens_t, slots = attend_case(bd, lens, 1, 2, 32, 16, E4, BF)
    B = 4099
    pick = torch.arange(B) * 5 % len(lens)
    out, lse = run_attend(bd, c, q[pick].contiguous(), table[pick].contiguous(), lens_t[pick].contiguous())
    alone, alone_lse = run_attend(bd, c, q, table, lens_t)
    check_attend(c, q, lens, slots, alone, alone_lse, 32 ** -0.5)
    # a row may be cut elsewhere in another batch: two bf16 roundings and the sums' own
    o, a = ref.to64(out), ref.to64(alone)[pick.numpy()]
    assert np.all(np.abs(o - a) <= 2.0 ** -7 * np.abs(a) + 2.0 ** -14)


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_attend_scales(bd, scale):
    for kind in (BF, E4):
        lens = [1, 40, 400]
        c, q, table, lens_t, slots = attend_case(bd, lens, 2, 2, 64, 16, kind, BF, spread=3.0)
        out, lse = run_attend(bd, c, q, table, lens_t, scale)
        check_attend(c, q, lens, slots, out, lse, scale)


def test_attend_rising_scores(bd):
    """Scores that rise by far more than the running maximum's slack, token by token, and fall again."""
    lens = [600]
    for kind in (BF, E4):
        for up in (1, -1):
            c, q, table, lens_t, slots = attend_case(bd, lens, 1, 2, 64, 16, kind, BF)
            k = torch.zeros((600, 1, 64))
            k[:, 0, 0] = up * torch.arange(600).float()
            v = torch.randn((600, 1, 64), generator=gen_of(2))
            q = torch.zeros((1, 2, 64), dtype=BF)
            q[0, 0, 0], q[0, 1, 0] = 1.0, 0.125
            s = torch.tensor(slots, dtype=torch.int32)
            c.expect(k, v, s)
            bd.bd_kv_write(c.kv, k.to(DEV), v.to(DEV), s.to(DEV))
            out, lse = run_attend(bd, c, q, table, lens_t, 1.0)
            check_attend(c, q, lens, slots, out, lse, 1.0)


def test_attend_infinite_and_nan_rows(bd):
    """Infinities and NaN in a sequence's own rows act as in the formula and stay in their sequence."""
    lens = [70, 70, 70, 300, 3]
    c, q, table, lens_t, slots = attend_case(bd, lens, 1, 2, 32, 16, BF, BF)
    k = torch.randn((513, 1, 32), generator=gen_of(3)).to(BF)
    v = torch.randn((513, 1, 32), generator=gen_of(4)).to(BF)
    q = q.abs()
    k[5, 0, 0] = -float("inf")          # one score -infinity: the others carry on
    v[75, 0, 3] = float("inf")          # an infinite value: one infinite output
    k[150, 0, 1] = float("nan")         # NaN scores: a NaN row
    v[400, 0, 2] = float("nan")         # one NaN output
    k[510:513, 0, 0] = -float("inf")    # every score -infinity: NaN, as in the formula
    s = torch.tensor(slots, dtype=torch.int32)
    c.expect(k, v, s)
    bd.bd_kv_write(c.kv, k.to(DEV), v.to(DEV), s.to(DEV))
    out, lse = run_attend(bd, c, q, table, lens_t)
    o = ref.to64(out)
    check_attend(c, q, lens, slots, out, lse, 32 ** -0.5, rows=(0,))
    assert np.isposinf(o[1, :, 3]).all() and np.isfinite(np.delete(o[1], 3, 1)).all()
    assert np.isnan(o[2]).all() and np.isnan(o[4]).all()
    assert np.isnan(o[3, :, 2]).all() and np.isfinite(np.delete(o[3], 2, 1)).all()


def test_attend_pages_and_lengths_out_of_range(bd):
    """A bad page or length gives NaN in its own sequence and touches nothing else."""
    for kind in (BF, E4):
        lens = [200, 200, 200, 30, 1000, 50]
        c, q, table, lens_t, slots = attend_case(bd, lens, 2, 2, 64, 16, kind, BF)
        good, good_lse = run_attend(bd, c, q, table, lens_t)
        bad, bad_len = table.clone(), lens_t.clone()
        bad[1, 12] = -1                      # the last page in use
        bad[2, 0] = c.kv.num_pages
        bad[4, 40] = 2 ** 31 - 1
        bad_len[3] = -5
        bad_len[5] = table.shape[1] * 16 + 1
        out, lse = run_attend(bd, c, q, bad, bad_len)
        for b in (1, 2, 4, 5):
            assert out[b].isnan().all() and lse[b].isnan().all()
        assert (out[3] == 0).all() and (lse[3] == -float("inf")).all()
        check_attend(c, q, lens, slots, out, lse, 0.125, rows=(0,))


def test_attend_forms(bd):
    """Strided queries and tables, given outputs, an empty batch; nothing is written around the outputs."""
    lens = [33, 0, 140, 7]
    c, q, table, lens_t, slots = attend_case(bd, lens, 2, 4, 64, 16, E4, F32)
    out, lse = run_attend(bd, c, q, table, lens_t)
    wide = torch.full((4, 3 * 8 * 64), float("nan"), device=DEV)
    wide[:, 512:1024] = q.to(DEV).view(4, 512)
    wt = torch.full((4, table.shape[1] + 5), -7, dtype=torch.int32, device=DEV)
    wt[:, :table.shape[1]] = table.to(DEV)
    mem = torch.full((4 + 2, 8, 64), 3.5, dtype=BF, device=DEV)
    got = bd.bd_attend(wide[:, 512:1024].view(4, 8, 64), c.kv, wt[:, :table.shape[1]], lens_t.to(DEV), out=mem[1:5])
    assert same_bits(got, out) and (mem[0] == 3.5).all() and (mem[5] == 3.5).all()
    heads_first = q.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)
    assert same_bits(bd.bd_attend(heads_first, c.kv, table.to(DEV), lens_t.to(DEV)), out)
    assert bd.bd_attend(q[:0].to(DEV), c.kv, table[:0].to(DEV), lens_t[:0].to(DEV)).shape == (0, 8, 64)
    one = bd.bd_attend(q[2:3].to(DEV), c.kv, table[2:3].to(DEV), lens_t[2:3].to(DEV), lse=lse[2:3])
    check_attend(c, q[2:3], [140], slots[33:173], one, lse[2:3], 0.125)


def test_attend_outputs_apart_from_inputs(bd):
    lens = [33, 140]
    c, q, table, lens_t, _ = attend_case(bd, lens, 2, 4, 64, 16, BF, BF)
    args = (c.kv, table.to(DEV), lens_t.to(DEV))
    gq = q.to(DEV)
    with pytest.raises(ValueError, match="out overlaps q"):
        bd.bd_attend(gq, *args, out=gq)
    out = torch.empty_like(gq)
    with pytest.raises(ValueError, match="overlaps"):
        bd.bd_attend(gq, *args, out=out, lse=out.view(torch.float32).view(-1)[:16].view(2, 8))
    wide = torch.zeros((2, 16, 64), dtype=BF, device=DEV)
    with pytest.raises(ValueError, match="overlaps"):    # in the gaps of q's strides
        bd.bd_attend(wide[:, :8], *args, out=wide.view(-1)[512:1536].view(2, 8, 64))


def test_attend_through_the_c_abi(bd):
    """The C call with a workspace of just the size asked for, used again by the next call, and with one that is not
    needed: nothing is written around them."""
    import ctypes
    from tenant_serving_amd import step
    lib = step._library()
    for lens, page in (([100, 3], 16), ([1000, 129, 0], 16)):
        c, q, table, lens_t, slots = attend_case(bd, lens, 2, 2, 64, page, E4, BF)
        B, hq, D = q.shape
        gq, gt, gl = q.to(DEV), table.to(DEV), lens_t.to(DEV)
        need = lib.bd_attend_workspace_bytes(B, hq, 2, D, page, table.shape[1])
        assert (need == 0) == (table.shape[1] * page <= 384)
        mem = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device=DEV)
        out = torch.empty((B, hq, D), dtype=BF, device=DEV)
        lse = torch.empty((B, hq), dtype=F32, device=DEV)
        qs = step._Pair(hq * D, D)
        for _ in range(3):
            st = lib.bd_attend(c.kv._ref, gq.data_ptr(), 0, qs, hq, gt.data_ptr(), table.shape[1], table.shape[1],
                               gl.data_ptr(), B, D ** -0.5, out.data_ptr(), lse.data_ptr(), mem.data_ptr() + 4096,
                               need, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
            assert st == 0
            check_attend(c, q, lens, slots, out, lse, D ** -0.5)
        assert (mem[:4096] == 0xA5).all() and (mem[4096 + need:] == 0xA5).all()


@pytest.mark.parametrize("dim", [64, 80, 96, 112, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("kind", [BF, E4])
@pytest.mark.parametrize("q_t", [BF, F32])
def test_attend_dims(bd, dim, kind, q_t):
    """Every head size and type with more units than workgroups, in a workspace of just the size asked for, which knows
    no types: nothing is written around it.  Then rows of few units, which no two workgroups share."""
    import ctypes
    from tenant_serving_amd import step
    lib = step._library()
    for base, B, rows in (([1930, 97, 0, 700], 260, (0, 1, 2, 3, 131, 136, 259)), ([380, 61, 0, 129], 20, range(20))):
        print("attend dims", dim, kind, q_t, B, flush=True)
        c, q, table, lens_t, slots = attend_case(bd, base, 2, 3, dim, 16, kind, q_t, "tokens")
        # the base's sequences again and again, with the same pages
        pick = torch.arange(B) * 3 % 4
        first = np.concatenate([[0], np.cumsum(base)])
        lens = [base[i] for i in pick]
        slots = [t for i in pick for t in slots[first[i]:first[i + 1]]]
        q, table, lens_t = (q[pick] * torch.linspace(0.5, 1, B)[:, None, None]).to(q_t), table[pick], lens_t[pick]
        hq = q.shape[1]
        gq, gt, gl = q.to(DEV), table.to(DEV), lens_t.to(DEV)
        need = lib.bd_attend_workspace_bytes(B, hq, 2, dim, 16, table.shape[1])
        assert (need > 0) == (B == 260)
        mem = torch.full((need + (16 << 20),), 0xA5, dtype=torch.uint8, device=DEV)
        out = torch.empty((B, hq, dim), dtype=BF, device=DEV)
        lse = torch.empty((B, hq), dtype=F32, device=DEV)
        st = lib.bd_attend(c.kv._ref, gq.data_ptr(), step._IN[q_t], step._Pair(hq * dim, dim), hq, gt.data_ptr(),
                           table.shape[1], table.shape[1], gl.data_ptr(), B, dim ** -0.5, out.data_ptr(),
                           lse.data_ptr(), mem.data_ptr() + (8 << 20), need,
                           ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert st == 0
        check_attend(c, q, lens, slots, out, lse, dim ** -0.5, rows)
        assert (mem[:8 << 20] == 0xA5).all() and (mem[(8 << 20) + need:] == 0xA5).all()


@pytest.mark.parametrize("B,page", [(5, 16), (66, 16), (300, 8), (1 << 20, 8), ((1 << 20) + 5, 8)])
def test_attend_rows_in_one_piece(bd, B, page):
    """Rows that are not split: few and many, up to more of them than workgroups, among empty and one-token ones."""
    lens = [0, 1, 30, 64, 130, 7, 128, 129] if page == 16 else [0, 1, 8, 3]
    c, q, table, lens_t, slots = attend_case(bd, lens, 1, 2, 16, page, E4, BF)
    pick = torch.arange(B) * 5 % len(lens)
    out, lse = run_attend(bd, c, q[pick].contiguous(), table[pick].contiguous(), lens_t[pick].contiguous())
    alone, alone_lse = run_attend(bd, c, q, table, lens_t)
    check_attend(c, q, lens, slots, alone, alone_lse, 0.25)
    pick = pick.to(DEV)
    assert same_bits(out, alone[pick]) and same_bits(lse, alone_lse[pick])


@pytest.mark.parametrize("B,heads,dim,kind", [(256, 4, 16, BF), (65, 12, 64, E4), (130, 4, 96, BF)])
def test_attend_longest_first(bd, B, heads, dim, kind):
    """More rows in one piece than workgroups at a time, which take them by length: bad lengths among them too."""
    base = [0, 700, 1, 129, 300, 128, 2, 1023]
    c, q, table, lens_t, slots = attend_case(bd, base, heads, 1, dim, 8, kind, BF)
    first = np.concatenate([[0], np.cumsum(base)])
    pick = torch.arange(B) * 5 % 8
    lens = [base[i] for i in pick]
    slots = [t for i in pick for t in slots[first[i]:first[i + 1]]]
    given = lens_t[pick].clone()
    bad = list(range(7, B, 50))
    for i in bad:
        given[i] = 2 ** 31 - 1 if i % 100 == 7 else 1025
    out, lse = run_attend(bd, c, q[pick].contiguous(), table[pick].contiguous(), given)
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    fine = [i for i in range(B) if i not in bad]
    check_attend(c, q[pick], lens, slots, out, lse, dim ** -0.5, fine[:24] + fine[-8:])


def test_attend_fp32_queries_and_infinite_keys(bd):
    """fp32 queries against keys with infinities: a score of -infinity drops out, whatever the queries' second term."""
    lens = [70, 300]
    c, q, table, lens_t, slots = attend_case(bd, lens, 1, 2, 32, 16, BF, F32)
    k = torch.randn((370, 1, 32), generator=gen_of(3)).to(BF)
    v = torch.randn((370, 1, 32), generator=gen_of(4)).to(BF)
    q = q.abs() + 0.1
    k[5, 0, 0] = -float("inf")
    k[200, 0, 7] = -float("inf")
    s = torch.tensor(slots, dtype=torch.int32)
    c.expect(k, v, s)
    bd.bd_kv_write(c.kv, k.to(DEV), v.to(DEV), s.to(DEV))
    out, lse = run_attend(bd, c, q, table, lens_t)
    # where a score broke, the wave's queries are one bf16 term: half a step, 2^-8, of each
    at = 0
    for b, n in enumerate(lens):
        kr = np.stack([c.row64(0, x) for x in slots[at:at + n]])
        vr = np.stack([c.row64(1, x) for x in slots[at:at + n]])
        at += n
        want, want_lse, S = ref.attend(ref.to64(q)[b], kr, vr, 32 ** -0.5)
        ds = 2.0 ** -8 * S + 40 * U * S
        tol = 2.0 ** -8 * np.abs(want) + 2 * np.abs(vr).max() * (np.expm1(2 * ds) + 2.0 ** -8 + (n + 64) * U)
        assert np.all(np.abs(ref.to64(out)[b] - want) <= tol)
        assert np.all(np.abs(ref.to64(lse)[b] - want_lse) <= ds + 1e-4)


def test_offsets_past_32_bits(bd):
    """Rows at the far end of arrays of more than 4 GiB each."""
    heads, page, dim = 8, 16, 128
    pages = (1 << 32) // (heads * page * dim * 2) + 40
    kv = bd.bd_kv_cache.empty(pages, heads, page, dim, BF, DEV)
    n = 100
    used = torch.tensor([pages - 1, 0, pages - 17, pages // 2 + 3, 5, pages - 2, 77], dtype=torch.int32)
    pos = torch.arange(n)
    slots = used[pos // page] * page + (pos % page).to(torch.int32)
    k, v = rows_of(n, heads, dim, BF, 1), rows_of(n, heads, dim, BF, 2)
    bd.bd_kv_write(kv, k.to(DEV), v.to(DEV), slots.to(DEV))
    rk, rv = bd.bd_kv_read(kv, slots.to(DEV))
    assert same_bits(rk, k) and same_bits(rv, v)
    assert same_bits(kv.k[pages - 1, :, 3], k[3]) and same_bits(kv.v[pages - 17, :, 1], v[33])
    q = torch.randn((1, 16, dim), generator=gen_of(6)).to(BF)
    out = ref.to64(bd.bd_attend(q.to(DEV), kv, used[None].to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV)))
    want, _, S = ref.attend(ref.to64(q)[0], ref.to64(k), ref.to64(v), dim ** -0.5)
    vmax = np.abs(ref.to64(v)).max()
    tol = 2.0 ** -8 * np.abs(want) + 2 * vmax * (np.expm1(2 * (dim + 8) * U * S) + 2.0 ** -15 + (n + 64) * U)
    assert np.all(np.abs(out[0] - want) <= tol)


# ----------------------------------------------------------------------------
# streams, graphs, and the operators together

def test_streams(bd):
    """Calls on two streams at once, each with its own outputs, against the same calls one after the other."""
    lens = [900, 3, 257]
    cases = [attend_case(bd, lens, 2, 4, 64, 16, kind, BF, seed=s) for kind, s in ((E4, 1), (BF, 2))]
    args = [(q.to(DEV), c.kv, t.to(DEV), n.to(DEV)) for c, q, t, n, _ in cases]
    want = [bd.bd_attend(*a) for a in args]
    x, _, gain, _ = on_gpu(*norm_inputs(64, 2048, BF, None, BF, 1))
    normed = bd.bd_rms_norm(x, gain)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((bd.bd_attend(*args[i]), bd.bd_rms_norm(x, gain)))
    torch.cuda.synchronize()
    for i in range(2):
        for o, y in got[i]:
            assert same_bits(o, want[i]) and same_bits(y, normed)


def test_graph_of_a_step(bd):
    """Norm, write and attention captured once and replayed while lengths, slots and inputs change, with eager calls
    of other sizes between the replays."""
    B, heads, group, dim, page, most = 3, 2, 4, 64, 16, 30
    d = heads * group * dim
    for kind in (E4, BF):
        c = Cache(bd, B * most, heads, page, dim, kind)
        table = torch.randperm(B * most, generator=gen_of(1)).to(torch.int32).view(B, most).to(DEV)
        gain = torch.ones((1, d), dtype=BF, device=DEV)
        x, res = torch.zeros((B, d), device=DEV), torch.zeros((B, d), dtype=BF, device=DEV)
        k, v = (torch.zeros((B, heads, dim), device=DEV) for _ in range(2))
        lens, slots = (torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(2))

        def step():
            y, r = bd.bd_rms_norm(x, gain, residual=res)
            bd.bd_kv_write(c.kv, k, v, slots)
            return y, r, bd.bd_attend(y.view(B, heads * group, dim), c.kv, table, lens)

        side = torch.cuda.Stream()
        slots.fill_(-1)
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = step()
        gen = gen_of(7)
        start = [0, 100, 251]
        for t in range(8):
            n = [min(most * page, s + (t + 1)) for s in start] if t != 5 else [0, 1, 480]
            x.copy_(torch.randn((B, d), generator=gen))
            res.copy_(torch.randn((B, d), generator=gen))
            k.copy_(torch.randn((B, heads, dim), generator=gen))
            v.copy_(torch.randn((B, heads, dim), generator=gen))
            lens.copy_(torch.tensor(n))
            slots.copy_(torch.tensor([int(table[b, (m - 1) // page]) * page + (m - 1) % page if m else -1
                                      for b, m in enumerate(n)]))
            if t == 0:   # fill what the lengths take for granted
                every = torch.arange(c.slots, dtype=torch.int32, device=DEV)
                fill = torch.randn((2, c.slots, heads, dim), generator=gen).to(DEV)
                bd.bd_kv_write(c.kv, fill[0], fill[1], every)
            graph.replay()
            first = [h.clone() for h in held]
            bd.bd_attend(x.view(B, heads * group, dim)[:1], c.kv, table[:1], lens[:1])
            torch.cuda.synchronize()
            eager = step()
            for a, b in zip(first, eager):
                assert same_bits(a, b), t


def test_two_graphs_in_turn(bd):
    """Two captured calls, replayed in turn with eager ones between them, each with a workspace of its own."""
    cases = [attend_case(bd, lens, 2, 4, 64, 16, kind, BF, seed=s)
             for lens, kind, s in (([900, 3, 257], E4, 1), ([2000, 150], BF, 2))]
    args = [(q.to(DEV), c.kv, t.to(DEV), n.to(DEV)) for c, q, t, n, _ in cases]
    want = [bd.bd_attend(*a) for a in args]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for a in args:
            bd.bd_attend(*a)
    torch.cuda.synchronize()
    graphs, held = [], []
    for a in args:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            held.append(bd.bd_attend(*a))
        graphs.append(g)
    for _ in range(6):
        for h in held:
            h.fill_(7.0)
        graphs[0].replay()
        graphs[1].replay()
        again = bd.bd_attend(*args[0])
        graphs[0].replay()
        torch.cuda.synchronize()
        assert same_bits(held[0], want[0]) and same_bits(held[1], want[1]) and same_bits(again, want[0])


def test_tensors_of_another_device(bd, monkeypatch):
    """Where the current device is not the tensors', the call makes theirs current (told here that it is not)."""
    from tenant_serving_amd import step
    real, left = step._current_device, []

    def other_once():
        return left.pop() if left else real()
    monkeypatch.setattr(step, "_current_device", other_once)
    x, res, gain, ids = on_gpu(*norm_inputs(4, 64, BF, BF, BF, 2))
    c, q, table, lens, _ = attend_case(bd, [40, 9], 2, 2, 64, 16, BF, BF)
    slots = torch.arange(4, dtype=torch.int32, device=DEV)
    rows = torch.randn((4, 2, 64), generator=gen_of(1)).to(BF).to(DEV)
    calls = [lambda: bd.bd_rms_norm(x, gain, residual=res, variant_ids=ids)[0],
             lambda: bd.bd_rms_norm_e4m3(x, gain, variant_ids=ids)[0],
             lambda: bd.bd_attend(q.to(DEV), c.kv, table.to(DEV), lens.to(DEV)),
             lambda: (bd.bd_kv_write(c.kv, rows, rows, slots), bd.bd_kv_read(c.kv, slots)[1])[1]]
    for call in calls:
        want = call()
        left.append(1)
        assert same_bits(call(), want) and not left


def test_a_layer_together(bd):
    """Two tokens' worth of a small attention block: norm, the fused linears, write, attention, output linear, norm;
    each operator against its plain form on what the one before gave."""
    import oracle
    from tenant_serving_amd import synth
    d, hq, heads, dim, page, V = 512, 8, 2, 64, 16, 3
    gen = synth.generator(77, DEV)
    weights = {}
    for name, n in (("q", hq * dim), ("k", heads * dim), ("v", heads * dim), ("o", d)):
        w = synth.base_weight(gen, n, d, DEV)
        sets = [bd.bd_compress(synth.laplace_delta(gen, n, d, 1e-3, DEV), 1) for _ in range(V)]
        weights[name] = (w, [s for s, _ in sets], [a for _, a in sets])
    gains = (1 + 0.1 * torch.randn((2, V, d), generator=gen, device=DEV)).to(BF)

    def linear(name, x, ids):
        w, s, a = weights[name]
        y = bd.bd_linear_grouped(x, ids, w, s, a, 1)
        want = oracle.linear_grouped(x.cpu(), ids.cpu(), w.cpu(), [t.cpu().numpy() for t in s],
                                     [t.cpu().numpy() for t in a], True)
        err = ref.to64(y) - want
        assert np.linalg.norm(err) <= 1e-3 * np.linalg.norm(want)
        return y

    for kind in (E4, BF):
        c = Cache(bd, 12, heads, page, dim, kind)
        lens = [35, 50]
        ids = torch.tensor([2, 0], dtype=torch.int32, device=DEV)
        table = torch.tensor([[3, 9, 1, -1], [0, 7, 4, 11]], dtype=torch.int32)
        slots = [[int(table[b, t // page]) * page + t % page for t in range(n)] for b, n in enumerate(lens)]
        # the context of both sequences but their last token
        past = torch.tensor(slots[0][:-1] + slots[1][:-1], dtype=torch.int32)
        pk, pv = rows_of(len(past), heads, dim, BF, 1), rows_of(len(past), heads, dim, BF, 2)
        c.expect(pk, pv, past)
        bd.bd_kv_write(c.kv, pk.to(DEV), pv.to(DEV), past.to(DEV))
        x = torch.randn((2, d), generator=gen, device=DEV)
        res = torch.randn((2, d), generator=gen, device=DEV).to(BF)
        h, r1 = bd.bd_rms_norm(x, gains[0], residual=res, variant_ids=ids)
        want, res_want = ref.rms_norm(x, gains[0], 1e-5, res, ids)
        check_bf16(h, want, d)
        assert same_bits(r1, res_want)
        q, k, v = (linear(n, h, ids) for n in ("q", "k", "v"))
        new = torch.tensor([s[-1] for s in slots], dtype=torch.int32)
        c.expect(k.cpu().view(2, heads, dim), v.cpu().view(2, heads, dim), new)
        bd.bd_kv_write(c.kv, k.view(2, heads, dim), v.view(2, heads, dim), new.to(DEV))
        c.check()
        qs = q.view(2, hq, dim)
        out, lse = run_attend(bd, c, qs, table, torch.tensor(lens, dtype=torch.int32))
        check_attend(c, qs, lens, slots[0] + slots[1], out, lse, dim ** -0.5)
        y = linear("o", out.view(2, d), ids)
        h2, r2 = bd.bd_rms_norm(y, gains[1], residual=r1, variant_ids=ids, residual_out=r1)
        want, _ = ref.rms_norm(y, gains[1], 1e-5, res_want, ids)
        check_bf16(h2, want, d)
        assert r2 is r1
