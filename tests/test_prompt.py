"""Attention of a prompt's tokens: refusals on the host, and GPU parity with the plain 64-bit form of
tests/more_reference.py.

Tolerances (u = 2^-24): a score is off by at most ds (more_reference.score_error), a weight by a factor exp(2 ds) and by
half a step of bf16, 2^-8 of itself; so an output is off by 2^-8 of itself as it is stored, by 2^-8 of the weights' mean of
|v|, and by expm1(2 ds) + (n + 64) u of the largest |v| twice.  The roundings of the weights are independent of each other:
over all outputs of a case the errors' root mean square is below that of 2^-8 / sqrt(3) of every term and of the result
(the standard deviation of an error that is even within half a step) and of what is left of the other bound."""

import ctypes

import numpy as np
import pytest
import torch

import tenant_serving_amd as bd
from tenant_serving_amd import prompt, step
from tests import more_reference as ref
from tests import test_attend_formed as formed

DEV = "cuda:0"
U = 2.0 ** -24
BF, F32, E4, E2 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.float4_e2m1fn_x2
FAKE = 1 << 20
same_bits, gen_of, rows64 = formed.same_bits, formed.gen_of, formed.rows64


# ----------------------------------------------------------------------------
# on the host

def test_c_refusals():
    lib = step._library()
    for kind, strides in ((0, (2048, 1024, 64)), (2, (2048, 1024, 64)), (4, (1024, 512, 32))):
        kv = step._KV(FAKE, FAKE, FAKE, FAKE, kind, 2, 64, 16, 10, *strides)
        need = lib.bd_attend_prompt_workspace_bytes(5, 2, 4, 2, 64, 16, 100)
        assert need > 0

        def call(form=None, **c):
            a = dict(kv=ctypes.byref(kv), q=FAKE, qs=step._Pair(256, 64), heads=4, T=5, table=FAKE, stride=100, pages=100,
                     lengths=FAKE, starts=FAKE, B=2, scale=0.125, scores=None, out=FAKE, lse=FAKE, ws=FAKE, bytes=need,
                     stream=None)
            if form is not None:
                a["scores"] = ctypes.byref(step._Scores(*form))
            a.update(c)
            return lib.bd_attend_prompt(*a.values())
        for form, want in [((float("nan"), None, None, None), 2), ((-1.0, None, None, None), 2), ((2.0 ** 61, None, None, None), 2),
                           ((0.0, FAKE + 2, None, None), 3), ((0.0, None, FAKE + 1, None), 3), ((0.0, None, None, FAKE + 3), 3)]:
            assert call(form) == want, form
        for change, want in [(dict(kv=None), 1), (dict(q=None), 1), (dict(qs=None), 1), (dict(table=None), 1),
                             (dict(lengths=None), 1), (dict(starts=None), 1), (dict(out=None), 1), (dict(T=-1), 2),
                             (dict(T=(1 << 27) + 1), 2), (dict(B=-1), 2), (dict(B=(1 << 21) + 1), 2), (dict(heads=0), 2),
                             (dict(heads=3), 2), (dict(heads=65538), 2), (dict(pages=0), 2), (dict(pages=(1 << 20) + 1), 2),
                             (dict(stride=-1), 2), (dict(scale=float("inf")), 2), (dict(scale=float("nan")), 2),
                             (dict(qs=step._Pair(-8, 64)), 2), (dict(qs=step._Pair(260, 64)), 3),
                             (dict(q=FAKE + 2), 3), (dict(out=FAKE + 2), 3), (dict(table=FAKE + 2), 3),
                             (dict(lengths=FAKE + 2), 3), (dict(starts=FAKE + 2), 3), (dict(lse=FAKE + 2), 3),
                             (dict(ws=None), 4), (dict(bytes=need - 4), 4), (dict(ws=FAKE + 8), 4)]:
            assert call(**change) == want, change
        empty = dict(q=None, table=None, lengths=None, starts=None, out=None, ws=None, bytes=0)
        assert call(T=0, **empty) == 0 and call(B=0, **empty) == 0
    for bad in [(0, 2, 4, 2, 64, 16, 9), (5, 0, 4, 2, 64, 16, 9), (5, 2, 3, 2, 64, 16, 9), (5, 2, 4, 2, 72, 16, 9),
                (5, 2, 4, 2, 64, 12, 9), (5, 2, 4, 2, 64, 16, 0), (5, 2, 4, 2, 64, 16, 1 << 21)]:
        assert lib.bd_attend_prompt_workspace_bytes(*bad) == 0
    assert lib.bd_attend_prompt_workspace_bytes(5, 2, 4, 2, 64, 16, 8) == 0        # too short a table to split


def test_binding_refusals(monkeypatch):
    with monkeypatch.context() as m:
        m.setattr(step, "_same_gpu", lambda device, named: None)
        kv = bd.bd_kv_cache.empty(6, 2, 16, 64, BF, "cpu")
    kv._dev = 0
    q, table = torch.zeros((5, 4, 64), dtype=BF), torch.zeros((3, 2), dtype=torch.int32)
    lens, starts = torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    five, slopes, big = torch.zeros(5, dtype=torch.int32), torch.zeros(4), torch.zeros(4096)
    out = kv.k.view(-1)[:1280].view(5, 4, 64)
    for err, match, args, kw in [
            (TypeError, "kv", (q, None, table, lens, starts), {}), (TypeError, "bfloat16", (q.float(), kv, table, lens, starts), {}),
            (TypeError, "q must be", (q.double(), kv, table, lens, starts), {}), (ValueError, "q must be", (q[0], kv, table, lens, starts), {}),
            (ValueError, "q must be", (torch.zeros((5, 4, 80), dtype=BF), kv, table, lens, starts), {}),
            (ValueError, "multiple of the cache", (q[:, :3], kv, table, lens, starts), {}),
            (TypeError, "page_table", (q, kv, table.long(), lens, starts), {}), (ValueError, "page_table", (q, kv, table[0], lens, starts), {}),
            (ValueError, "page_table", (q, kv, table[:, :0], lens, starts), {}),
            (ValueError, "contiguous", (q, kv, torch.zeros((2, 3), dtype=torch.int32).t(), lens, starts), {}),
            (ValueError, "2\\^24", (q, kv, torch.zeros((3, (1 << 20) + 1), dtype=torch.int32), lens, starts), {}),
            (ValueError, "lengths", (q, kv, table, lens[:2], starts), {}), (ValueError, "starts", (q, kv, table, lens, starts[:3]), {}),
            (TypeError, "starts", (q, kv, table, lens, starts.long()), {}), (ValueError, "scale", (q, kv, table, lens, starts), dict(scale=2.0 ** 61)),
            (ValueError, "cap", (q, kv, table, lens, starts), dict(cap=0.0)), (TypeError, "slopes", (q, kv, table, lens, starts), dict(slopes=slopes.double())),
            (ValueError, "slopes", (q, kv, table, lens, starts), dict(slopes=slopes[:3])), (ValueError, "first", (q, kv, table, lens, starts), dict(first=lens)),
            (TypeError, "last", (q, kv, table, lens, starts), dict(last=five.float())), (TypeError, "out", (q, kv, table, lens, starts), dict(out=q.float())),
            (ValueError, "lse", (q, kv, table, lens, starts), dict(lse=torch.zeros(5, 3))), (ValueError, "out overlaps q", (q, kv, table, lens, starts), dict(out=q)),
            (ValueError, "out overlaps the cache", (q, kv, table, lens, starts), dict(out=out)),
            (ValueError, "lse overlaps first", (q, kv, table, lens, starts), dict(first=big.view(torch.int32)[10:15], lse=big[:20].view(5, 4))),
            (ValueError, "lse overlaps starts", (q, kv, table, lens, big.view(torch.int32)[19:23]), dict(lse=big[:20].view(5, 4))),
            (ValueError, "GPU", (q, kv, table, lens, starts), dict(cap=30.0, slopes=slopes, first=five, last=five))]:
        with pytest.raises(err, match=match):
            bd.bd_attend_prompt(*args, **kw)


def test_reference():
    """The plain prompt form against the plain form of one token, row by row."""
    rng = np.random.default_rng(5)
    q, k, v = rng.standard_normal((4, 6, 16)), rng.standard_normal((9, 2, 16)), rng.standard_normal((9, 2, 16))
    slopes = rng.random(6)
    out, lse, _, mean, share = ref.attend_prompt(q, k, v, 0.3, [0, 2, 5, 7], [6, 9, 5, 30], [5, 6, 7, 8], 2.0, slopes)
    for t, (a, b, pos) in enumerate(((0, 6, 5), (2, 9, 6), (5, 5, 7), (7, 30, 8))):
        want, want_lse, _ = ref.attend(q[t], k, v, 0.3, 2.0, slopes, a, b, pos)
        assert np.allclose(out[t], want, atol=1e-12) and np.allclose(lse[t], want_lse, atol=1e-12)
    assert (out[2] == 0).all() and (lse[2] == -np.inf).all() and (share <= mean + 1e-12).all()


# ----------------------------------------------------------------------------
# on the GPU

def case(new, past, heads, group, dim, page, kind, layout="heads", seed=21, fix=None):
    """Sequences of new[b] tokens behind past[b], over a cache whose other places hold random bytes, NaN among them."""
    lens = [a + b for a, b in zip(new, past)]
    c, _, table, lengths, slots = formed.case(lens, heads, group, dim, page, kind, BF, layout, seed, fix=fix)
    T = sum(new)
    q = (torch.randn((T, heads * group, dim), generator=gen_of(seed + 1)) * 2).to(BF)
    starts = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
    return c, q, table, lengths, starts, slots


def run(c, q, table, lengths, starts, **kw):
    lse = torch.full(q.shape[:2], 7.0, dtype=F32, device=DEV)
    out = torch.full(q.shape, 7.0, dtype=BF, device=DEV)
    kw = {n: x.to(DEV) if isinstance(x, torch.Tensor) else x for n, x in kw.items()}
    got = bd.bd_attend_prompt(q.to(DEV), c.kv, table.to(DEV), lengths.to(DEV), starts.to(DEV), out=out, lse=lse, **kw)
    assert got is out
    return out, lse


def check(c, q, starts, slots, out, lse, scale=None, cap=None, slopes=None, first=None, last=None, only=None, some=None):
    """some: of each sequence's new tokens only these are looked at."""
    dim = q.shape[2]
    scale = dim ** -0.5 if scale is None else scale
    out, lse, q64 = (t.cpu().double().numpy() for t in (out, lse, q))
    slope = None if slopes is None else slopes.double().numpy()
    square = count = 0.0
    for b, own in enumerate(slots):
        s0, s1 = int(starts[b]), int(starts[b + 1])
        n = len(own)
        t = np.arange(s0, s1)
        if some is not None:
            t = t[[i for i in some if -(s1 - s0) <= i < s1 - s0]]
        if (only is not None and b not in only) or not len(t):
            continue
        pos = n - s1 + t
        lo = np.zeros(len(t), int) if first is None else first.numpy()[t]
        hi = pos + 1 if last is None else last.numpy()[t]
        kr, vr = (rows64(c, i, own) if n else np.zeros((0, c.heads, dim)) for i in (0, 1))
        want, want_lse, S, mean, share = ref.attend_prompt(q64[t], kr, vr, scale, lo, hi, pos, cap or 0.0, slope)
        far = np.maximum(np.abs(pos), n).max(initial=0)
        ds = ref.score_error(dim, S, cap or 0.0, 0.0 if slope is None else S + np.abs(slope).max() * far)
        fine = np.abs(vr[np.isfinite(vr)])
        rest = 2 * fine.max(initial=0.0) * (np.expm1(2 * ds) + (n + 64) * U) + 2.0 ** -133
        tol = 2.0 ** -8 * (np.abs(want) + mean) + rest
        o = out[t]
        assert np.array_equal(np.isnan(o), np.isnan(want)), (b, np.argwhere(np.isnan(o) != np.isnan(want))[:4].tolist())
        with np.errstate(invalid="ignore"):
            near = (np.abs(o - want) <= tol) | (o == want) | np.isnan(want)
            assert near.all(), (b, np.argwhere(~near)[:4].tolist(), np.nanmax(np.abs(o - want)))
            sigma = np.sqrt(4.0 ** -8 / 3 * (want ** 2 + share ** 2) + rest ** 2)
            ok = np.isfinite(want)
            square += ((o - want)[ok] ** 2 / sigma[ok] ** 2).sum()
            count += ok.sum()
        okl = np.isfinite(want_lse)
        assert np.array_equal(lse[t][~okl], want_lse[~okl], equal_nan=True)
        tl = ds + (n + 64) * U + 4 * U * np.abs(want_lse[okl])
        assert np.all(np.abs(lse[t][okl] - want_lse[okl]) <= tl), (b, n)
    assert count == 0 or square / count <= 1.0 + 4 / np.sqrt(count), (square / count, count)


NEW = [1, 2, 5, 16, 17, 31, 32, 33, 0, 64, 65, 100, 129]
PAST = [0, 63, 64, 1, 7, 200, 95, 33, 40, 0, 191, 130, 5]


@pytest.mark.gpu
@pytest.mark.parametrize("kind,dims", [(BF, (16, 48, 64, 80, 96, 128, 176, 192, 256)), (E4, (16, 64, 80, 96, 128, 192, 208, 256)),
                                       (E2, (32, 64, 96, 128, 160, 192, 224, 256))])
def test_sizes(kind, dims):
    for dim in dims:
        for heads, group, page, layout in ((2, 4, 16, "heads"), (1, 3, 24, "tokens")):
            print("prompt", kind, dim, heads, group, flush=True)
            c, q, table, lengths, starts, slots = case(NEW, PAST, heads, group, dim, page, kind, layout)
            out, lse = run(c, q, table, lengths, starts)
            check(c, q, starts, slots, out, lse, some=(0, 1, 2, 30, 31, 32, 33, 63, 64, -2, -1))


@pytest.mark.gpu
@pytest.mark.parametrize("heads,group", [(1, 1), (3, 1), (1, 8), (2, 16), (1, 17), (2, 33), (1, 130), (9, 2)])
def test_head_layouts(heads, group):
    print("prompt heads", heads, group, flush=True)
    for kind, dim, page in ((BF, 64, 8), (E2, 128, 48)):
        new, past = [5, 40, 1, 0, 130], [3, 0, 200, 9, 64]
        c, q, table, lengths, starts, slots = case(new, past, heads, group, dim, page, kind, "both")
        out, lse = run(c, q, table, lengths, starts)
        check(c, q, starts, slots, out, lse, some=(0, 1, 31, 32, 127, 128, -1))


@pytest.mark.gpu
@pytest.mark.parametrize("new,past", [([5], [5000]), ([1, 2, 3], [3000, 10, 700]), ([130], [2500]), ([3] * 9, [900] * 9),
                                      ([257, 1], [1100, 4000]), ([16] * 3, [0, 6000, 20])])
@pytest.mark.parametrize("kind", [BF, E4, E2])
def test_splits(new, past, kind):
    """Few rows behind long contexts: a tile's keys in several workgroups, and none left for some of them."""
    print("prompt split", new, past, kind, flush=True)
    c, q, table, lengths, starts, slots = case(new, past, 2, 4, 64, 16, kind)
    assert prompt._prompt_bytes(q.shape[0], len(new), 8, 2, 64, 16, table.shape[1]) > 0
    out, lse = run(c, q, table, lengths, starts)
    check(c, q, starts, slots, out, lse, some=(0, 1, 31, 32, 129, -1))
    again, lse2 = run(c, q, table, lengths, starts)
    assert same_bits(out, again) and same_bits(lse, lse2)


def ranges(kind, new, past, seed=2):
    """first and last of every new token, by the kind of mask."""
    rng = np.random.default_rng(seed)
    first, last = [], []
    for n, p in zip(new, past):
        pos = np.arange(p, p + n)
        f, l = np.zeros(n, int), pos + 1
        if kind == "window":
            f = pos - rng.integers(0, 90)
        elif kind == "documents":
            f = pos // 37 * 37
        elif kind == "prefix":
            l = np.maximum(pos + 1, (p + n) // 2)
        elif kind == "both":
            f, l = pos - 20, pos + 21
        elif kind == "any":
            f, l = rng.integers(-5, p + n + 5, n), rng.integers(-5, p + n + 9, n)
        elif kind == "nothing":
            f = np.where(np.arange(n) % 3 == 0, pos + 1, 0)
            l = np.where(np.arange(n) % 5 == 1, -2 ** 31, l)
            f = np.where(np.arange(n) // 32 == 1, 2 ** 31 - 1, f)
        first.append(f)
        last.append(l)
    return [torch.tensor(np.concatenate(x), dtype=torch.int32) for x in (first, last)]


@pytest.mark.gpu
@pytest.mark.parametrize("mask", ["window", "documents", "prefix", "both", "any", "nothing"])
@pytest.mark.parametrize("kind", [BF, E4, E2])
def test_masks(mask, kind):
    new, past = [1, 33, 0, 150, 7, 70], [100, 64, 3, 0, 400, 31]
    first, last = ranges(mask, new, past)
    for dim, heads, group in ((64, 2, 3), (128, 1, 1), (192, 1, 4), (96, 2, 1)):
        print("prompt mask", mask, kind, dim, flush=True)
        c, q, table, lengths, starts, slots = case(new, past, heads, group, dim, 16, kind)
        out, lse = run(c, q, table, lengths, starts, first=first, last=last)
        check(c, q, starts, slots, out, lse, first=first, last=last)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [BF, E4, E2])
def test_formed_scores(kind):
    new, past = [1, 33, 0, 130, 7], [1100, 64, 3, 0, 400]
    for dim, heads, group in ((64, 2, 3), (128, 1, 8), (256, 1, 2), (96, 1, 1), (160, 1, 2)):
        slopes = torch.exp2(-4 * torch.rand(heads * group, generator=gen_of(1))) * torch.where(torch.arange(heads * group) % 5 == 4, -0.01, 1.0)
        first, last = ranges("both", new, past)
        for kw in (dict(cap=3.0), dict(slopes=slopes), dict(cap=50.0, slopes=slopes, first=first, last=last, scale=-0.7), dict(scale=-0.2),
                   dict(cap=1e4, first=first)):
            print("prompt formed", kind, dim, sorted(kw), flush=True)
            c, q, table, lengths, starts, slots = case(new, past, heads, group, dim, 16, kind)
            out, lse = run(c, q, table, lengths, starts, **kw)
            check(c, q, starts, slots, out, lse, some=(0, 1, 5, 31, 32, 100, -1), **kw)


@pytest.mark.gpu
def test_scores_of_any_size():
    new, past = [40, 3], [30, 600]
    for kind in (BF, E4, E2):
        c, q, table, lengths, starts, slots = case(new, past, 2, 2, 64, 16, kind)
        for scale in (0.0, 2.0 ** 60, -2.0 ** 40, 2.0 ** 20, 1e-30):
            kw = dict(scale=scale)
            out, lse = run(c, q, table, lengths, starts, **kw)
            o = out.cpu().double().numpy()
            assert np.isfinite(o).all()
            if abs(scale) <= 1:
                check(c, q, starts, slots, out, lse, **kw)
            else:       # the largest score's token alone
                s0 = int(starts[1])
                for t in (s0, s0 + 2):
                    kr, vr = (rows64(c, i, slots[1]) for i in (0, 1))
                    for h in range(4):
                        s = (kr[:601 + t - s0, h // 2] @ q[t, h].double().numpy()) * np.sign(scale)
                        top = np.argsort(s)
                        if abs(scale) * (s[top[-1]] - s[top[-2]]) > 1000 + abs(scale) * 80 * U * np.abs(s[top[-1]]) * 40:
                            assert np.all(np.abs(o[t, h] - vr[top[-1], h // 2]) <= 2.0 ** -8 * np.abs(vr[top[-1], h // 2]))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [BF, E4, E2])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
def test_what_is_not_seen_does_not_matter(kind, dim):
    """NaN and infinities in rows of the sequence that some of its tokens see and others do not: only those get them."""
    new, past = [130, 70], [0, 500]
    at = [3, 20, 64, 100, 129, 130 + 10, 130 + 505, 130 + 569]

    def fix(k, v):
        for i, j in enumerate(at):
            x = (float("nan"), float("inf"), -float("inf"))[i % 3]
            v[j, :, i * 5 % v.shape[2]] = x
            if i % 2:
                v[j, :, 1] = -x
            if i % 4 == 3:
                k[j] = x
    c, q, table, lengths, starts, slots = case(new, past, 2, 3, dim, 16, kind, fix=fix)
    first, last = ranges("both", new, past)
    seen = run(c, q, table, lengths, starts)
    check(c, q, starts, slots, *seen)
    out, lse = run(c, q, table, lengths, starts, first=first, last=last)
    check(c, q, starts, slots, out, lse, first=first, last=last)
    bad = ~out.isfinite().all(2).all(1).cpu()
    tokens = torch.arange(200)
    pos = torch.where(tokens < 130, tokens, tokens + 370)
    for j in range(200):
        mine = [x - 130 if j >= 130 else x for x in at if (x >= 130) == (j >= 130)]
        assert bool(bad[j]) == any(int(pos[j]) - 20 <= x < int(pos[j]) + 21 for x in mine), j
    for kw in (dict(cap=5.0), dict(slopes=torch.full((6,), 0.05))):
        out, lse = run(c, q, table, lengths, starts, first=first, last=last, **kw)
        check(c, q, starts, slots, out, lse, first=first, last=last, **kw)


@pytest.mark.gpu
def test_pages_lengths_and_starts_out_of_range():
    for kind in (BF, E4, E2):
        new, past = [6, 6, 6, 6, 6, 0], [34, 34, 34, 34, 34, 10]
        c, q, table, lengths, starts, slots = case(new, past, 2, 2, 64, 8, kind)
        table[0, 1], table[1, 0], table[2, 4] = 10 ** 6, -1, -5
        first = torch.zeros(30, dtype=torch.int32)
        first[6:12] = torch.tensor([7, 8, 9, 15, 16, 0])        # of sequence 1, only the first and last see page 0
        lengths[3], lengths[4] = 41, -3
        out, lse = run(c, q, table, lengths, starts, first=first)
        nan = out.cpu().isnan().all(2).all(1)
        assert torch.equal(nan, out.cpu().isnan().any(2).any(1)) and torch.equal(nan, lse.cpu().isnan().any(1))
        # sequence 2 sees page 4 (tokens 32 ..) from every one of its tokens
        want = [True] * 6 + [True, False, False, False, False, True] + [True] * 6 + [True] * 6 + [False] * 6
        assert nan.tolist() == want
        assert (out[24:] == 0).all() and (lse[24:] == -float("inf")).all()
        check(c, q, starts[1:3], slots[1:2], out, lse, first=first, some=(1, 2, 3, 4))
    # starts past the ends, rows outside them, and more new tokens than the sequence has
    c, q, table, lengths, starts, slots = case([9, 20, 11], [5, 0, 60], 2, 2, 64, 16, BF)
    want, want_lse = run(c, q, table, lengths, starts)
    less = starts.clone()
    less[0], less[3] = 4, 35
    lengths2 = lengths.clone()
    lengths2[2] -= 5
    out, lse = run(c, q, table, lengths2, less)
    assert (out[:4] == 7).all() and (out[35:] == 7).all() and (lse[:4] == 7).all() and (lse[35:] == 7).all()
    assert same_bits(out[9:29], want[9:29]) and same_bits(lse[9:29], want_lse[9:29])
    check(c, q, torch.tensor([4, 9]), slots[:1], out, lse)
    check(c, q, torch.tensor([29, 35]), [slots[2][:66]], out, lse)
    wide = starts.clone()
    wide[0], wide[3] = -100, 2 ** 31 - 1
    out, lse = run(c, q, table, lengths, wide)
    assert same_bits(out, want)
    out, lse = run(c, q, table, torch.tensor([3, 20, 71], dtype=torch.int32), starts)      # the first six come before it
    assert (out[:6] == 0).all() and (lse[:6] == -float("inf")).all()
    check(c, q, torch.tensor([6, 9]), [slots[0][:3]], out, lse)
    down = torch.tensor([9, 0, 29, 40], dtype=torch.int32)      # a falling number: no tokens for the first
    out, lse = run(c, q, table, lengths, down)
    assert same_bits(out[29:], want[29:])


@pytest.mark.gpu
def test_many_sequences():
    """Hundreds of ragged sequences, more than a wave has lanes and than the GPU has workgroups."""
    rng = np.random.default_rng(4)
    new = rng.integers(0, 20, 400).tolist()
    past = rng.integers(0, 60, 400).tolist()
    c, q, table, lengths, starts, slots = case(new, past, 2, 3, 32, 8, E4)
    out, lse = run(c, q, table, lengths, starts)
    check(c, q, starts, slots, out, lse, only=range(0, 400, 7))
    new = [0] * 5000
    new[17], new[4999], new[300] = 3, 5, 40
    c, q, table, lengths, starts, slots = case(new, [1] * 5000, 1, 2, 64, 8, BF)
    out, lse = run(c, q, table, lengths, starts)
    check(c, q, starts, slots, out, lse, only=(17, 300, 4999))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [BF, E4, E2])
def test_a_long_prompt(kind):
    """A prompt of more tiles than workgroups at a time, rows from all over it."""
    c, q, table, lengths, starts, slots = case([2500, 700], [0, 1800], 4, 4, 128, 32, kind)
    out, lse = run(c, q, table, lengths, starts)
    check(c, q, starts, slots, out, lse, some=tuple(range(3, 2500, 311)) + (-1,))


@pytest.mark.gpu
def test_one_new_token_is_what_attend_gives():
    for kind in (BF, E4, E2):
        past = [0, 7, 300, 2000, 64]
        c, q, table, lengths, starts, slots = case([1] * 5, past, 2, 4, 128, 16, kind)
        first = torch.tensor([0, 3, 100, 1000, 64], dtype=torch.int32)
        slopes = torch.rand(8, generator=gen_of(3)) * 0.1
        for kw in (dict(), dict(cap=20.0, slopes=slopes, first=first)):
            out, lse = run(c, q, table, lengths, starts, **kw)
            check(c, q, starts, slots, out, lse, **kw)
            one, one_lse = formed.run(c, q, table, lengths, **kw)
            formed.check(c, q, slots, one, one_lse, **kw)


@pytest.mark.gpu
def test_strided_queries_and_tables():
    c, q, table, lengths, starts, slots = case([20, 33], [64, 3], 2, 3, 80, 16, BF)
    want, _ = run(c, q, table, lengths, starts)
    wide = torch.zeros((53, 9, 96), dtype=BF, device=DEV)
    wide[:, 1:7, 8:88] = q.to(DEV)
    tables = torch.full((2, table.shape[1] + 5), -1, dtype=torch.int32, device=DEV)
    tables[:, :table.shape[1]] = table.to(DEV)
    heads_out = q.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)
    for x, t in ((wide[:, 1:7, 8:88], tables[:, :table.shape[1]]), (heads_out, table.to(DEV))):
        assert same_bits(bd.bd_attend_prompt(x, c.kv, t, lengths.to(DEV), starts.to(DEV)), want)
    none = bd.bd_attend_prompt(q[:0].to(DEV), c.kv, table.to(DEV), lengths.to(DEV), torch.zeros(3, dtype=torch.int32, device=DEV))
    assert none.shape == (0, 6, 80)
    bd.bd_attend_prompt(q.to(DEV), c.kv, table[:0].to(DEV), lengths[:0].to(DEV), starts[:1].to(DEV))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Keys and values, and queries, past 4 GiB of their arrays."""
    heads, page, dim, n = 8, 16, 128, 100
    pages = (1 << 32) // (heads * page * dim * 2) + 40
    kv = bd.bd_kv_cache.empty(pages, heads, page, dim, BF, DEV)
    used = torch.tensor([pages - 1, 0, pages - 17, pages // 2 + 3, 5, pages - 2, 77], dtype=torch.int32)
    pos = torch.arange(n)
    slots = used[pos // page] * page + (pos % page).to(torch.int32)
    k, v = (torch.randn((n, heads, dim), generator=gen_of(s)).to(BF) for s in (1, 2))
    bd.bd_kv_write(kv, k.to(DEV), v.to(DEV), slots.to(DEV))
    base = torch.empty(2 * (1 << 30) + 4096, dtype=BF, device=DEV)
    q = torch.as_strided(base, (3, 16, dim), (1 << 30, dim, 1))
    x = torch.randn((3, 16, dim), generator=gen_of(6)).to(BF)
    q.copy_(x.to(DEV))
    out = bd.bd_attend_prompt(q, kv, used[None].to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV), torch.tensor([0, 3], dtype=torch.int32, device=DEV))
    want, _, S, mean, _ = ref.attend_prompt(x.double().numpy(), k.double().numpy(), v.double().numpy(), dim ** -0.5, [0] * 3, [98, 99, 100], [97, 98, 99])
    tol = 2.0 ** -8 * (np.abs(want) + mean) + 2 * v.abs().max().item() * (np.expm1(2 * ref.score_error(dim, S)) + (n + 64) * U)
    assert np.all(np.abs(out.cpu().double().numpy() - want) <= tol)


@pytest.mark.gpu
def test_streams_graphs_and_devices(monkeypatch):
    new, past = [5, 130], [900, 70]
    cases = [case(new, past, 2, 2, 64, 16, kind, seed=s) for kind, s in ((E2, 1), (BF, 2))]
    dev = [(q.to(DEV), c.kv, t.to(DEV), n.to(DEV), st.to(DEV)) for c, q, t, n, st, _ in cases]
    first, last = (x.to(DEV) for x in ranges("both", new, past))
    kw = dict(cap=30.0, slopes=torch.full((4,), 0.1, device=DEV), first=first, last=last)
    want = [bd.bd_attend_prompt(*a, **kw) for a in dev]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(bd.bd_attend_prompt(*dev[i], **kw))
    torch.cuda.synchronize()
    assert all(same_bits(o, want[i]) for i in range(2) for o in got[i])
    graphs, held = [torch.cuda.CUDAGraph() for _ in range(2)], [None, None]
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g):
            held[i] = bd.bd_attend_prompt(*dev[i], **kw)
    for i in range(3):
        first.add_(3)
        dev[0][3].sub_(1)
        dev[1][0].copy_(torch.randn(dev[1][0].shape, generator=gen_of(i)))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for j in range(2):
            assert same_bits(held[j], bd.bd_attend_prompt(*dev[j], **kw))
    real, left = step._current_device, [1]
    monkeypatch.setattr(step, "_current_device", lambda: left.pop() if left else real())
    assert same_bits(bd.bd_attend_prompt(*dev[0], **kw), held[0]) and not left
