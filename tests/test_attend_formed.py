"""Attention of one new token with formed scores (a cap, a bias by distance, a first token) and over the 4-bit cache:
refusals on the host, and GPU parity with the plain 64-bit form of tests/more_reference.py.

Tolerances: as in test_step_gpu.py, with the score's error from more_reference.score_error; fp32 queries enter as three
bf16 terms that hold them whole."""

import ctypes

import numpy as np
import pytest
import torch

import tenant_serving_amd as bd
from tenant_serving_amd import step
from tests import more_reference as ref
from tests import test_cache_four as four
from tests import test_step_gpu as eight

DEV = "cuda:0"
U = 2.0 ** -24
BF, F32, E4, E2 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float4_e2m1fn_x2
FAKE = 1 << 20
same_bits, gen_of = eight.same_bits, eight.gen_of


# ----------------------------------------------------------------------------
# on the host

def test_c_refusals():
    lib = step._library()
    for kind, strides in ((2, (2048, 1024, 64)), (4, (1024, 512, 32))):
        kv = step._KV(FAKE, FAKE, FAKE, FAKE, kind, 2, 64, 16, 10, *strides)
        need = lib.bd_attend_workspace_bytes(2, 4, 2, 64, 16, 100)

        def call(form=None, **c):
            a = dict(kv=ctypes.byref(kv), q=FAKE, q_type=0, qs=step._Pair(256, 64), heads=4, table=FAKE, stride=100,
                     pages=100, lengths=FAKE, B=2, scale=0.125, scores=None, out=FAKE, lse=FAKE, ws=FAKE, bytes=need,
                     stream=None)
            if form is not None:
                a["scores"] = ctypes.byref(step._Scores(*form))
            a.update(c)
            return lib.bd_attend_scores(*a.values())
        for form, want in [((float("nan"), None, None, None), 2), ((-1.0, None, None, None), 2),
                           ((float("inf"), None, None, None), 2), ((2.0 ** 61, None, None, None), 2),
                           ((2.0 ** -61, None, None, None), 2), ((0.0, FAKE + 2, None, None), 3),
                           ((0.0, None, FAKE + 1, None), 3), ((0.0, None, None, FAKE), 5)]:
            assert call(form) == want, form
        good = (30.0, FAKE, FAKE, None)
        for change, want in [(dict(kv=None), 1), (dict(q=None), 1), (dict(out=None), 1), (dict(lengths=None), 1),
                             (dict(q_type=2), 5), (dict(heads=3), 2), (dict(ws=None), 4), (dict(bytes=need - 4), 4),
                             (dict(pages=0), 2), (dict(B=-1), 2)]:
            assert call(good, **change) == want, change
        assert call(good, B=0, q=None, table=None, lengths=None, out=None, ws=None, bytes=0) == 0


def test_binding_refusals(monkeypatch):
    with monkeypatch.context() as m:
        m.setattr(step, "_same_gpu", lambda device, named: None)
        kv = bd.bd_kv_cache.empty(6, 2, 16, 64, E2, "cpu")
    kv._dev = 0
    q, table = torch.zeros((3, 4, 64), dtype=BF), torch.zeros((3, 2), dtype=torch.int32)
    lens, slopes = torch.zeros(3, dtype=torch.int32), torch.zeros(4)
    for err, match, kw in [(ValueError, "cap", dict(cap=0.0)), (ValueError, "cap", dict(cap=-1.0)),
                           (ValueError, "cap", dict(cap=float("nan"))), (ValueError, "cap", dict(cap=2.0 ** 61)),
                           (TypeError, "slopes", dict(slopes=slopes.double())), (ValueError, "slopes", dict(slopes=slopes[:3])),
                           (TypeError, "first", dict(first=lens.long())), (ValueError, "first", dict(first=lens[:2])),
                           (ValueError, "GPU", dict(cap=30.0, slopes=slopes, first=lens))]:
        with pytest.raises(err, match=match):
            bd.bd_attend(q, kv, table, lens, **kw)
    one = torch.zeros(64)
    with pytest.raises(ValueError, match="lse overlaps slopes"):
        bd.bd_attend(q, kv, table, lens, slopes=one[8:12], lse=one[:12].view(3, 4))
    with pytest.raises(ValueError, match="lse overlaps first"):
        bd.bd_attend(q, kv, table, lens, first=one.view(torch.int32)[11:14], lse=one[:12].view(3, 4))


# ----------------------------------------------------------------------------
# on the GPU

def make_cache(kind, pages, heads, page, dim, layout, seed):
    if kind == E2:
        return four.Cache(pages, heads, page, dim, layout, seed)
    return eight.Cache(bd, pages, heads, page, dim, kind, layout, seed)


def rows64(c, which, slots):
    """What the cache holds at these slots: float64 [n, heads, dim]."""
    p, at = np.divmod(np.asarray(slots, int), c.page)
    r = c.rows[which][p, :, at]
    if isinstance(c, four.Cache):
        return ref.decode4(ref.unpack4(r), c.scales[which][p, :, :, at])
    if c.kind == E4:
        return eight.ref.decode(r, c.scales[which][p, :, at][..., None])
    wide = r[..., 0::2].astype(np.uint32) << 16 | r[..., 1::2].astype(np.uint32) << 24     # bf16 bits as fp32's upper half
    return wide.view(np.float32).astype(np.float64)


def case(lens, heads, group, dim, page, kind, q_t, layout="heads", seed=21, keep_from=None, fix=None):
    """A ragged batch over a cache whose other places hold random bytes, NaN among them.  keep_from: per sequence the
    first token attended to; pages with none from there on are not in the table."""
    gen = gen_of(seed)
    B, most = len(lens), max(1, max(-(-n // page) for n in lens))
    need = sum(-(-n // page) for n in lens) + 3
    c = make_cache(kind, need, heads, page, dim, layout, seed)
    order = torch.randperm(need, generator=gen).tolist()
    table = torch.full((B, most), -1, dtype=torch.int32)
    slots, write = [], []
    for b, n in enumerate(lens):
        for i in range(-(-n // page)):
            table[b, i] = order.pop()
        slots.append([int(table[b, t // page]) * page + t % page for t in range(n)])
        skip = max(0, keep_from[b]) if keep_from else 0
        write.append([s if t >= skip else -1 for t, s in enumerate(slots[b])])
        for i in range(min(skip, n) // page):
            table[b, i] = -7 if i % 2 else 1 << 30
    T = sum(lens)
    k, v = torch.randn((T, heads, dim), generator=gen).to(BF), torch.randn((T, heads, dim), generator=gen).to(BF)
    if fix:
        fix(k, v)
    q = (torch.randn((B, heads * group, dim), generator=gen) * 2).to(q_t)
    flat = torch.tensor(sum(write, []), dtype=torch.int32)
    if T:
        c.expect(k, v, flat)
        bd.bd_kv_write(c.kv, k.to(DEV), v.to(DEV), flat.to(DEV))
    return c, q, table, torch.tensor(lens, dtype=torch.int32), slots


def run(c, q, table, lens, **kw):
    lse = torch.empty(q.shape[:2], dtype=F32, device=DEV)
    kw = {n: x.to(DEV) if isinstance(x, torch.Tensor) else x for n, x in kw.items()}
    return bd.bd_attend(q.to(DEV), c.kv, table.to(DEV), lens.to(DEV), lse=lse, **kw), lse


def check(c, q, slots, out, lse, scale=None, cap=None, slopes=None, first=None, rows=None, loose=0.0):
    dim = q.shape[2]
    scale = dim ** -0.5 if scale is None else scale
    out, lse, q64 = (t.cpu().double().numpy() for t in (out, lse, q))
    slope = None if slopes is None else slopes.double().numpy()
    for b, own in enumerate(slots):
        if rows is not None and b not in rows:
            continue
        n = len(own)
        lo = 0 if first is None else min(max(0, int(first[b])), n)
        kr, vr = (rows64(c, i, own[lo:]) for i in (0, 1))
        want, want_lse, S = ref.attend(q64[b], kr, vr, scale, cap or 0.0, slope)
        ds = ref.score_error(dim, S, cap or 0.0, 0.0 if slope is None else S + np.abs(slope).max() * (n - lo)) + loose * S
        fine = np.abs(vr[np.isfinite(vr)])
        vmax = fine.max() if fine.size else 0.0
        tol = 2.0 ** -8 * np.abs(want) + 2 * vmax * (np.expm1(2 * ds) + 2.0 ** -15 + (n + 64) * U) + 2.0 ** -133
        assert np.array_equal(np.isnan(out[b]), np.isnan(want)), b
        ok = ~np.isnan(want)
        with np.errstate(invalid="ignore"):
            near = (np.abs(out[b] - want) <= tol) | (out[b] == want)
        assert near[ok].all(), (b, n, lo, np.abs(out[b] - want)[ok].max())
        okl = np.isfinite(want_lse)
        assert np.array_equal(lse[b][~okl], want_lse[~okl], equal_nan=True)
        tl = ds + (n + 64) * U + 4 * U * np.abs(want_lse[okl])
        assert np.all(np.abs(lse[b][okl] - want_lse[okl]) <= tl), (b, n, lo)


EDGES = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 160, 255, 256, 257, 300]


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("q_t", [BF, F32])
def test_four_bits(dim, q_t):
    print("attend e2m1", dim, q_t, flush=True)
    for heads, group, page, layout, lens in ((2, 4, 16, "heads", EDGES), (1, 8, 24, "tokens", EDGES), (2, 17, 8, "both", [5, 700, 0, 64]),
                                             (3, 1, 64, "heads", [2500, 3])):
        c, q, table, n, slots = case(lens, heads, group, dim, page, E2, q_t, layout)
        out, lse = run(c, q, table, n)
        assert out.dtype == BF and out.shape == q.shape
        check(c, q, slots, out, lse)
        again, lse2 = run(c, q, table, n)
        assert same_bits(out, again) and same_bits(lse, lse2)


FORMS = [dict(cap=3.0), dict(slopes=True), dict(first=True), dict(cap=50.0, slopes=True, first=True, scale=-0.7)]


def formed(form, q, lens, seed=3):
    gen = gen_of(seed)
    kw = dict(form)
    if "slopes" in kw:
        kw["slopes"] = torch.exp2(-4 * torch.rand(q.shape[1], generator=gen)) * torch.where(torch.arange(q.shape[1]) % 5 == 4, -0.01, 1.0)
    if "first" in kw:
        far = torch.rand(len(lens), generator=gen)
        kw["first"] = torch.tensor([[-5, 0, n - 1, n, n + 9, int(n * x), n - 8, n - 100][i % 8]
                                    for i, (n, x) in enumerate(zip(lens, far.tolist()))], dtype=torch.int32)
    return kw


@pytest.mark.gpu
@pytest.mark.parametrize("kind,dims", [(BF, (16, 64, 96, 128, 192, 256)), (E4, (16, 80, 128, 176, 192, 256)), (E2, (32, 64, 96, 128, 192, 256))])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_forms(kind, dims, form):
    for dim in dims:
        for q_t in (BF, F32):
            print("attend formed", kind, dim, form, q_t, flush=True)
            lens = EDGES + [700, 1201, 2000]
            for heads, group, page, layout in ((2, 3, 16, "heads"), (1, 17, 24, "tokens")):
                shape = torch.empty((len(lens), heads * group, dim))
                kw = formed(FORMS[form], shape, lens)
                c, q, table, n, slots = case(lens, heads, group, dim, page, kind, q_t, layout,
                                             keep_from=kw["first"].tolist() if "first" in kw else None)
                out, lse = run(c, q, table, n, **kw)
                check(c, q, slots, out, lse, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [BF, E4, E2])
def test_windows_of_long_sequences(kind):
    """Windows much shorter than the sequences, split rows and rows in one piece, none of the pages before in the table;
    more sequences than workgroups, and than a wave has lanes."""
    for lens, window in (([9000, 40, 5000, 0, 2500, 128, 1], 1000), ([7 * i % 600 for i in range(300)], 77),
                         ([3000] * 9, 2000), ([350] * 70, 9)):
        first = torch.tensor([n - window for n in lens], dtype=torch.int32)
        c, q, table, n, slots = case(lens, 2, 2, 64, 16, kind, BF, keep_from=first.tolist())
        out, lse = run(c, q, table, n, first=first, cap=20.0)
        check(c, q, slots, out, lse, first=first, cap=20.0, rows=range(0, len(lens), 1 + len(lens) // 40))


@pytest.mark.gpu
def test_first_of_every_place():
    """A first token at every place of the first 140 and around the ends of pages and units."""
    lens = [300] * 140 + [1, 8, 9]
    first = torch.tensor(list(range(140)) + [0, 7, 8], dtype=torch.int32)
    for kind, page in ((BF, 8), (E4, 24), (E2, 16)):
        c, q, table, n, slots = case(lens, 1, 2, 32, page, kind, BF, keep_from=first.tolist())
        out, lse = run(c, q, table, n, first=first)
        check(c, q, slots, out, lse, first=first)


@pytest.mark.gpu
def test_masked_places_do_not_matter():
    """NaN and infinities before the first token, in its own group of 8, in keys and values."""
    lens, first = [200, 77, 1500], torch.tensor([101, 76, 1300], dtype=torch.int32)

    def fix(k, v):
        at = 0
        for n, f in zip(lens, first.tolist()):
            for i, x in enumerate((float("nan"), float("inf"), -float("inf"))):
                k[at + f - 1 - i], v[at + f - 1 - i] = x, x
            at += n
    for kind in (BF, E4, E2):
        for kw in (dict(), dict(cap=5.0), dict(slopes=torch.full((6,), 0.1))):
            c, q, table, n, slots = case(lens, 2, 3, 64, 16, kind, BF, fix=fix)
            out, lse = run(c, q, table, n, first=first, **kw)
            assert out.isfinite().all() and lse.isfinite().all()
            check(c, q, slots, out, lse, first=first, **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("q_t", [BF, F32])
def test_infinite_rows_and_large_scores(q_t):
    """Infinite keys are capped like any score; infinite values reach what sees them; scores far past the cap."""
    lens = [40, 300, 3000]

    def fix(k, v):
        k[3, :, :] = float("inf")
        k[50, :, 5] = -float("inf")
        v[60, 0, 7], v[400, 1, 3] = float("inf"), -float("inf")
        k[700] *= 3e4
    c, q, table, n, slots = case(lens, 2, 2, 64, 16, BF, q_t, fix=fix)      # codes hold no infinities
    q[0] = q[0].abs() + 0.25    # all products of the wholly infinite key have one sign
    out, lse = run(c, q, table, n, cap=8.0)
    # where a wave meets infinite keys its fp32 queries enter as one bf16 term, off by half a step, 2^-8 of each value:
    # a score by that part of its terms' magnitudes
    check(c, q, slots, out, lse, cap=8.0, loose=2.0 ** -8 if q_t == F32 else 0.0)
    for kind in (BF, E4, E2):
        c, q, table, n, slots = case(lens, 2, 2, 64, 16, kind, q_t, seed=5)
        for cap, scale in ((2.0 ** -60, 1.0), (1e-3, 1.0), (2.0 ** 60, 0.125), (1e6, 0.125), (100.0, 2.0 ** 60), (1.0, 0.0)):
            out, lse = run(c, q, table, n, cap=cap, scale=scale)
            check(c, q, slots, out, lse, cap=cap, scale=scale)


@pytest.mark.gpu
def test_pages_and_lengths_out_of_range():
    for kind in (BF, E2):
        c, q, table, n, slots = case([40, 40, 40, 40, 40], 2, 2, 64, 8, kind, BF)
        first = torch.tensor([0, 16, 24, 50, 0], dtype=torch.int32)
        table[0, 1], table[1, 1], table[2, 4] = 10 ** 6, -1, -5     # sequence 1 does not see its bad page
        n[3], n[4] = 41, -3
        out, lse = run(c, q, table, n, first=first)
        good = torch.zeros(5, dtype=torch.bool)
        good[1] = good[4] = True
        assert torch.equal(out.cpu().isnan().any(2).any(1), ~good) and torch.equal(out.cpu().isnan().all(2).all(1), ~good)
        assert (out[4] == 0).all() and (lse[4] == -float("inf")).all()
        check(c, q, slots, out, lse, first=first, rows=(1,))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """4-bit rows and scale bytes at the far end of arrays of more than 4 GiB."""
    heads, page, dim, n = 8, 16, 128, 100
    pages = (1 << 32) // (heads * page * dim // 2) + 40
    kv = bd.bd_kv_cache.empty(pages, heads, page, dim, E2, DEV)
    used = torch.tensor([pages - 1, 0, pages - 17, pages // 2 + 3, 5, pages - 2, 77], dtype=torch.int32)
    pos = torch.arange(n)
    slots = used[pos // page] * page + (pos % page).to(torch.int32)
    k, v = four.rows_of(n, heads, dim, BF, 1), four.rows_of(n, heads, dim, BF, 2)
    bd.bd_kv_write(kv, k.to(DEV), v.to(DEV), slots.to(DEV))
    q = torch.randn((1, 16, dim), generator=gen_of(6)).to(BF)
    out = bd.bd_attend(q.to(DEV), kv, used[None].to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV))
    k64, v64 = (ref.decode4(*ref.quantise4(x.double().numpy())) for x in (k, v))
    want, _, S = ref.attend(q[0].double().numpy(), k64, v64, dim ** -0.5)
    tol = 2.0 ** -8 * np.abs(want) + 2 * np.abs(v64).max() * (np.expm1(2 * (dim + 8) * U * S) + 2.0 ** -15 + (n + 64) * U)
    assert np.all(np.abs(out[0].cpu().double().numpy() - want) <= tol)


@pytest.mark.gpu
def test_streams_graphs_and_devices(monkeypatch):
    lens = [900, 3, 257]
    slopes, first = torch.tensor([0.1, 0.2, 0.3, 0.4]), torch.tensor([100, 0, 200], dtype=torch.int32)
    cases = [case(lens, 2, 2, 64, 16, kind, BF, seed=s) for kind, s in ((E2, 1), (E4, 2))]
    dev = [(q.to(DEV), c.kv, t.to(DEV), n.to(DEV)) for c, q, t, n, _ in cases]
    kw = dict(cap=30.0, slopes=slopes.to(DEV), first=first.to(DEV))
    want = [bd.bd_attend(*a, **kw) for a in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(bd.bd_attend(*dev[i], **kw))
    torch.cuda.synchronize()
    assert all(same_bits(o, want[i]) for i in range(2) for o in got[i])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = bd.bd_attend(*dev[0], **kw)
    for i in range(3):
        kw["first"].add_(40)
        dev[0][3].sub_(1)
        dev[0][0].copy_(torch.randn(dev[0][0].shape, generator=gen_of(i)))
        graph.replay()
        torch.cuda.synchronize()
        assert same_bits(held, bd.bd_attend(*dev[0], **kw))
    real, left = step._current_device, [1]
    monkeypatch.setattr(step, "_current_device", lambda: left.pop() if left else real())
    assert same_bits(bd.bd_attend(*dev[0], **kw), held) and not left


@pytest.mark.gpu
def test_given_outputs():
    c, q, table, n, slots = case([40, 300], 2, 2, 64, 16, E2, BF)
    first = torch.tensor([3, 100], dtype=torch.int32)
    want, lse = run(c, q, table, n, first=first)
    out = torch.empty_like(q, device=DEV)
    got = bd.bd_attend(q.to(DEV), c.kv, table.to(DEV), n.to(DEV), out=out, first=first.to(DEV))
    assert got is out and same_bits(out, want)
    with pytest.raises(ValueError, match="out overlaps the cache"):
        bd.bd_attend(q.to(DEV), c.kv, table.to(DEV), n.to(DEV), out=c.kv.k.view(BF).view(-1)[:q.numel()].view(q.shape), first=first.to(DEV))
    none = torch.empty((0, 4, 64), dtype=BF, device=DEV)
    assert bd.bd_attend(none, c.kv, table[:0].to(DEV), n[:0].to(DEV), cap=1.0).shape == (0, 4, 64)
