"""Attention of a prompt's tokens where a call's sizes or numbers are extreme: what tests/test_prompt.py leaves out.  Tolerances
as there, where none is derived beside a test."""

import numpy as np
import pytest
import torch

import tenant_serving_amd as bd
from tests import test_prompt as plain

DEV = "cuda:0"
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def tiles_found(starts, group, rows, most, grid):
    """What the kernels find for a grid's tiles, in whole numbers: for each (sequence, row), or None past the last one.
    The sum of a lane's sequences stops at `most`."""
    B = len(starts) - 1
    per = (B + 63) // 64
    n = np.maximum(np.diff(starts.astype(np.int64)), 0)
    tiles = (n * group + rows - 1) // rows
    sums = [0] * 64
    for lane in range(64):
        for t in tiles[lane * per:lane * per + per]:
            sums[lane] = min(sums[lane] + int(t), most)
    ends = np.cumsum(sums)
    assert ends[-1] < 1 << 31
    found = []
    for f in grid:
        if f >= ends[-1]:
            found.append(None)
            continue
        at = int(ends[-1]) - 1 - f
        lane = int(np.argmax(ends > at))
        at -= int(ends[lane]) - sums[lane]
        b = lane * per
        while at >= tiles[b] and b + 1 < B:
            at -= int(tiles[b])
            b += 1
        found.append((b, at * rows))
    return found


@pytest.mark.parametrize("B,T,group", [(70000, 1 << 25, 16), (70000, 1 << 19, 16), (1 << 18, 1 << 21, 16)])
def test_falling_starts_find_rows_of_their_sequence(B, T, group):
    """Sequences that all claim every token: their tiles pass 2^31, and each one found is still one of its sequence's."""
    starts = np.arange(B + 1) % 2 * T
    grid = [0, 1, T * group // 128 - 1, T * group // 128, T * group // 128 + B - 1] + list(range(5, T * group // 128 + B, 99991))
    for b, row in tiles_found(starts, group, 128, 1 << 24, grid):
        assert b % 2 == 0 and 0 <= row < T * group
    rising = np.sort(np.random.default_rng(1).integers(0, T + 1, 1001))
    tiles = (np.diff(rising) * group + 127) // 128
    want = [(b, r * 128) for b, t in enumerate(tiles) for r in range(t)][::-1]
    pick = [i for i in (0, 1, 100, len(want) // 3, len(want) - 1)]
    assert tiles_found(rising, group, 128, 1 << 24, pick + [len(want)]) == [want[i] for i in pick] + [None]


@pytest.mark.gpu
def test_sequences_that_claim_the_same_tokens():
    """Falling starts, so many that a lane's tiles pass what it sums them up to: every row holds its result or what was
    there, and nothing beside the rows is touched.  All sequences see the same three keys, so that it does not matter
    whose result a row has."""
    B, T, heads, dim, pad = 70000, 500000, 16, 16, 1 << 16
    kv = bd.bd_kv_cache.empty(1, 1, 8, dim, BF, DEV)
    k, v = (torch.randn((3, 1, dim), generator=plain.gen_of(s)).to(BF).to(DEV) for s in (1, 2))
    bd.bd_kv_write(kv, k, v, torch.arange(3, dtype=torch.int32, device=DEV))
    gen = torch.Generator(device=DEV).manual_seed(3)
    room = torch.full((T * heads * dim + 2 * pad,), float("nan"), dtype=BF, device=DEV)
    q = room[pad:-pad].view(T, heads, dim)
    q.copy_(torch.randn(q.shape, generator=gen, device=DEV))
    to = torch.full_like(room, 7.0)
    out = to[pad:-pad].view(T, heads, dim)
    starts = (torch.arange(B + 1, device=DEV) % 2 * T).to(torch.int32)
    table = torch.zeros((B, 1), dtype=torch.int32, device=DEV)
    lengths = torch.full((B,), 3, dtype=torch.int32, device=DEV)
    last = torch.full((T,), 3, dtype=torch.int32, device=DEV)
    print("falling starts", flush=True)
    bd.bd_attend_prompt(q, kv, table, lengths, starts, last=last, out=out)
    assert (to[:pad] == 7).all() and (to[-pad:] == 7).all()
    s = (q.view(-1, dim).double() @ k[:, 0].double().t().contiguous()) * dim ** -0.5
    p = torch.softmax(s, 1)
    want = (p @ v[:, 0].double()).view(T, heads, dim)
    mean = (p @ v[:, 0].double().abs()).view(T, heads, dim)
    reach = ((q.view(-1, dim).double().abs() @ k[:, 0].double().abs().t().contiguous()) * dim ** -0.5).max().item()
    ds = (dim + 8) * U * reach
    tol = 2.0 ** -8 * (want.abs() + mean) + 2 * v.abs().max().item() * (np.expm1(2 * ds) + 67 * U)
    left = (out == 7).all(2)
    near = ((out.double() - want).abs() <= tol).all(2)
    assert (near | left).all()
    assert near.any()


def lone_scores(kind, cap, new, past, seed=31):
    """A case whose scores are one exact product each, up to about twice the cap and of either sign: queries and keys are
    zero but in one column."""
    def fix(k, v):
        x = k[..., 5].clone()
        k.zero_()
        k[..., 5] = x
    c, q, table, lengths, starts, slots = plain.case(new, past, 2, 4, 64, 16, kind, seed=seed, fix=fix)
    x = q[..., 5].clone()
    q.zero_()
    q[..., 5] = x
    return c, q, table, lengths, starts, slots, cap / 2


def check_lone(lse, q, keys, cap, scale):
    """lse [n, heads] of rows that see one key each, keys [n, kv heads, dim]: it is the capped score.  Where the score before
    the cap is at most half of it: two roundings of the factor and of its product with the score, a polynomial of relative
    error 2^-25.7 whose last sum is rounded once and the roundings within it a third of one, a product with the cap and the
    sum's logarithm of an exponential and its own (4 u).  Beyond, tanh x = 1 - 2 / (1 + e^(2 x)): off by 8 u, as the
    exponential's argument is rounded, 2 x of its own size, which the slope of the whole at most halves, and the exponential,
    the inverse and the sums take a step each."""
    s = (q[..., 5] * keys[..., 5].repeat(q.shape[1] // keys.shape[1], 1)) * scale
    want = cap * np.tanh(s / cap)
    tol = np.where(np.abs(s) <= cap / 2 * (1 - 4 * U), 6 * U * np.abs(want), 8 * U * cap + 3 * U * np.abs(want)) + 4 * U
    off = np.abs(lse - want) / tol
    assert (off <= 1).all(), (cap, off.max(), (s / cap)[off > 1][:4])


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [BF, plain.E4, plain.E2])
@pytest.mark.parametrize("cap", [50.0, 1e4, 1e6, 2.0 ** 40])
def test_capped_scores_are_those_of_fp32(kind, cap):
    """Each token sees its own key only, so lse is its score: in a prompt, and as one new token of a sequence."""
    new, past = [200, 33, 1], [3, 64, 700]
    c, q, table, lengths, starts, slots, scale = lone_scores(kind, cap, new, past)
    pos = np.concatenate([np.arange(p, p + n) for n, p in zip(new, past)])
    first = torch.tensor(pos, dtype=torch.int32)
    keys = np.concatenate([plain.rows64(c, 0, own[p:]) for own, p in zip(slots, past)])
    values = np.concatenate([plain.rows64(c, 1, own[p:]) for own, p in zip(slots, past)])
    out, lse = plain.run(c, q, table, lengths, starts, scale=scale, cap=cap, first=first)
    q64, want = q.double().numpy(), values.repeat(4, 1)
    check_lone(lse.cpu().double().numpy(), q64, keys, cap, scale)
    assert (np.abs(out.cpu().double().numpy() - want) <= 2.0 ** -8 * 2 * np.abs(want)).all()     # its one weight is rounded too
    lens = torch.tensor(pos + 1, dtype=torch.int32)
    tables = torch.cat([table[b:b + 1].repeat(n, 1) for b, n in enumerate(new)])
    for x in (q, q.float()):
        out, lse = plain.formed.run(c, x, tables, lens, scale=scale, cap=cap, first=first)
        check_lone(lse.cpu().double().numpy(), q64, keys, cap, scale)
        assert np.array_equal(out.cpu().double().numpy(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [BF, plain.E2])
def test_slopes_far_above_the_cap(kind):
    """Slopes that over the cap leave fp32's range: at no distance they take nothing off, at any other everything."""
    new, past = [70, 3], [3, 64]
    c, q, table, lengths, starts, slots = plain.case(new, past, 2, 4, 64, 16, kind)
    pos = np.concatenate([np.arange(p, p + n) for n, p in zip(new, past)])
    values = np.concatenate([plain.rows64(c, 1, own[p:]) for own, p in zip(slots, past)]).repeat(4, 1)
    tables = torch.cat([table[b:b + 1].repeat(n, 1) for b, n in enumerate(new)])
    slopes = torch.full((8,), 2.0 ** 100)
    for cap in (2.0 ** -60, 2.0 ** -30, 1.0, None):
        kw = dict(slopes=slopes, cap=cap)
        out, lse = plain.run(c, q, table, lengths, starts, **kw)
        one, one_lse = plain.formed.run(c, q, tables, torch.tensor(pos + 1, dtype=torch.int32), **kw)
        for o, l in ((out, lse), (one, one_lse)):
            # a lone weight: exact, or rounded to bf16 as the result is
            assert (np.abs(o.cpu().double().numpy() - values) <= 2.0 ** -8 * 2 * np.abs(values)).all()
            assert l.isfinite().all() and (cap is None or (l.abs() <= cap + 4 * U).all())


# every width's kernels, whole and in part; formed scores of codes take four waves at 192 columns, eight at 96 and 128
@pytest.mark.gpu
@pytest.mark.parametrize("kind,dims", [(BF, (48, 80, 112, 192, 176, 224)), (plain.E4, (48, 80, 112, 192, 176, 224)),
                                       (plain.E2, (32, 192, 224))])
def test_formed_scores_of_every_width(kind, dims):
    new, past = [1, 33, 0, 130, 7], [1100, 64, 3, 0, 400]
    first, last = plain.ranges("both", new, past)
    for dim, (heads, group) in zip(dims, ((2, 3), (1, 8), (1, 1), (2, 4), (1, 2), (3, 1))):
        slopes = torch.exp2(-4 * torch.rand(heads * group, generator=plain.gen_of(1)))
        for kw in (dict(cap=3.0), dict(slopes=slopes), dict(cap=50.0, slopes=slopes, first=first, last=last, scale=-0.7)):
            print("prompt formed", kind, dim, sorted(kw), flush=True)
            c, q, table, lengths, starts, slots = plain.case(new, past, heads, group, dim, 16, kind)
            out, lse = plain.run(c, q, table, lengths, starts, **kw)
            plain.check(c, q, starts, slots, out, lse, some=(0, 1, 5, 31, 32, 100, -1), **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("kind,dim,kw", [(BF, 64, {}), (BF, 128, {}), (BF, 192, {}), (BF, 256, {}), (plain.E4, 96, {}), (plain.E4, 128, {}),
                                         (plain.E4, 256, {}), (plain.E2, 64, {}), (plain.E2, 128, dict(cap=20.0)), (plain.E2, 192, {}),
                                         (plain.E2, 192, dict(cap=20.0))])
def test_more_than_two_rounds_of_page_numbers(kind, dim, kw):
    """Workgroups that go over more than 128 tiles of keys, whose pages they look up 64 tiles at a time; also with pages
    that are not there, in each round, which only some tokens see."""
    keys, heads, group, n = (64 if dim <= 128 else 32), 2, 16, 2048
    past = 129 * keys + 40
    c, q, table, lengths, starts, slots = plain.case([n], [past], heads, group, dim, 16, kind)
    # nothing is split, so that a workgroup's tiles are all of a row's
    assert plain.prompt._prompt_bytes(n, 1, heads * group, heads, dim, 16, table.shape[1]) == 0 and past // keys > 128
    some = (0, 1, 31, 32, 127, 128, 900, 2040, -1)
    print("prompt rounds", kind, dim, kw, flush=True)
    out, lse = plain.run(c, q, table, lengths, starts, **kw)
    plain.check(c, q, starts, slots, out, lse, some=some, **kw)
    bad = [70 * keys + 3, 63 * keys, 128 * keys + 17]      # tokens whose pages are not there
    for i, j in enumerate(bad):
        table[0, j // 16] = (10 ** 6, -1, 2 ** 31 - 1)[i]
    sees = torch.arange(n) // 8 % 5
    first, last = torch.zeros(n, dtype=torch.int32), torch.zeros(n, dtype=torch.int32)
    ranges = [(0, 63 * keys), (63 * keys + 16, 70 * keys), (71 * keys, 128 * keys), (129 * keys, past), (0, past)]
    for i, (a, b) in enumerate(ranges):
        first[sees == i], last[sees == i] = a, b
    out, lse = plain.run(c, q, table, lengths, starts, first=first, last=last, **kw)
    nan = out.cpu().isnan().all(2).all(1)
    assert torch.equal(nan, sees == 4) and torch.equal(out.cpu().isnan().any(2).any(1), nan)
    assert torch.equal(lse.cpu().isnan().any(1), nan)
    some = [t for t in (0, 8, 16, 24, 31, 40, 127, 800, 808, 2040) if sees[t] < 4]
    plain.check(c, q, starts, slots, out, lse, first=first, last=last, some=some, **kw)


def formed_bound(q, k, scale, cap):
    """Capped scores [Hq, n] of q [Hq, D] and k [Hq, n, D] (float64), and how far one is off at most: the products' and
    sums' roundings as far as the cap lets them through, and 8 u of the cap (see check_lone).  The kernels' sums of
    infinite terms of one sign are exact."""
    with np.errstate(all="ignore"):
        prod = q[:, None, :] * k * scale
        s, a = prod.sum(2), np.abs(prod).sum(2)
        e = np.where(np.isfinite(a), (q.shape[1] + 8) * U * a, 0.0)
        through = np.where(np.isfinite(a), cap * (np.tanh((np.abs(s) + e) / cap) - np.tanh((np.abs(s) - e) / cap)), 0.0)
    return cap * np.tanh(s / cap), np.minimum(through, e).max() + 8 * U * cap


@pytest.mark.gpu
@pytest.mark.parametrize("q_t", [BF, F32])
@pytest.mark.parametrize("kind", [BF, plain.E4, plain.E2])
def test_scores_far_past_the_cap(kind, q_t):
    """Saturated scores, of finite and infinite keys, with bounds that a wrong one passes: a prompt's last tokens, and one
    new token.  fp32 queries hold bf16 values, as where a sequence's keys are infinite only these enter, and weights as one
    term like a prompt's."""
    lens, new, alone = [40, 300, 3000], 3, 2.0 ** -8 if kind == BF and q_t == F32 else 2.0 ** -15

    def fix(k, v):
        # a key's values have one sign, so that no score is what is left of larger terms
        k.copy_(k.abs() * torch.where(torch.arange(len(k)) % 3 == 0, 1, -1)[:, None, None])
        if kind == BF:
            k[3], k[350] = float("inf"), -float("inf")      # codes hold no infinities
        k[45] *= 3e4
        k[700] *= 3e4
        k[2000, 1] *= -1e5
    for cap, scale in ((8.0, 0.125), (100.0, 2.0 ** 60), (2.0 ** -20, -1.0), (30.0, -50.0)):
        c, q, table, lengths, starts, slots = plain.case([new] * 3, [n - new for n in lens], 2, 2, 64, 16, kind, fix=fix)
        q = q.abs() + 0.25          # all products of a wholly infinite key have one sign
        print("capped", kind, q_t, cap, scale, flush=True)
        out, lse = plain.run(c, q, table, lengths, starts, cap=cap, scale=scale)
        one, one_lse = plain.formed.run(c, q[new - 1::new].to(q_t).contiguous(), table, lengths, cap=cap, scale=scale)
        for b, own in enumerate(slots):
            k, v = (plain.rows64(c, i, own).transpose(1, 0, 2).repeat(2, 0) for i in (0, 1))
            for o, l, extra in ((out[b * new + new - 1], lse[b * new + new - 1], 2.0 ** -8), (one[b], one_lse[b], alone)):
                s, ds = formed_bound(q[b * new + new - 1].double().numpy(), k, scale, cap)
                p = np.exp(s - s.max(1, keepdims=True))
                want = (p[:, None] @ v)[:, 0] / p.sum(1)[:, None]
                mean = (p[:, None] @ np.abs(v))[:, 0] / p.sum(1)[:, None]
                n = len(own)
                tol = 2.0 ** -8 * np.abs(want) + extra * mean + 2 * np.abs(v).max() * (np.expm1(2 * ds) + (n + 64) * U)
                assert tol.max() < 0.1 * np.abs(v).max(), tol.max()      # or the test says nothing
                assert (np.abs(o.cpu().double().numpy() - want) <= tol).all(), (b, extra)
                want_lse = s.max(1) + np.log(p.sum(1))
                tl = ds + (n + 64) * U + 4 * U * np.abs(want_lse)
                assert tl.max() < 0.01 * max(1.0, cap) and (np.abs(l.cpu().double().numpy() - want_lse) <= tl).all(), (b, extra)
