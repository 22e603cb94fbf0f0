"""GPU parity of the attention of one new token where the call's form matters: page tables with far more columns than
the lengths need, as a serving program keeps them (rows are split then and joined, whatever their lengths), beside
tables just wide enough (rows stay in one piece); and scores of any size.  The plain implementation and the tolerances
are those of test_step_gpu.py unless a test derives its own."""

import numpy as np
import pytest
import torch

from tests import step_reference as ref
from tests.test_step_gpu import (BF, DEV, E4, EDGES, F32, U, attend_case, bd, check_attend, gen_of,  # noqa: F401
                                 run_attend, same_bits)

pytestmark = pytest.mark.gpu


def widened(table, page, tokens=4096):
    """The table with room for this many tokens per sequence; no page behind the last one in use."""
    more = max(0, tokens // page - table.shape[1])
    return torch.nn.functional.pad(table, (0, more), value=-1)


def is_split(c, q, table):
    """Whether the call lays out partial results, which it does exactly where rows may be split."""
    from tenant_serving_amd import step
    return step._library().bd_attend_workspace_bytes(q.shape[0], q.shape[1], c.heads, q.shape[2], c.kv.page_size,
                                                     table.shape[1]) > 0


@pytest.mark.parametrize("scale", [2.0 ** 10, 2.0 ** 25, 2.0 ** 31, -2.0 ** 40, 2.0 ** 60, -2.0 ** 60])
@pytest.mark.parametrize("wide", [False, True])
def test_large_scores(bd, scale, wide):
    """Scores of any size.  Queries and keys are small whole numbers, so that every q.k is a whole number held exactly:
    two scores are equal or 2^10 apart at least, and a weight is 1 or 0.  What is left are the sums of the values
    (n u each), the division and the output's rounding."""
    lens = [1, 40, 300, 129]
    for kind in (BF, E4):
        for factor in (1.0, 2.0 ** 50):      # the second: large by the keys, at a scale of 2^-50 of the given one
            for q_t in (BF, F32):
                print("large scores", scale, wide, kind, factor, q_t, flush=True)
                c, q, table, lens_t, slots = attend_case(bd, lens, 2, 2, 64, 16, kind, q_t)
                table = widened(table, 16) if wide else table
                assert is_split(c, q, table) == wide
                T, gen = len(slots), gen_of(9)
                k = torch.randint(-8, 9, (T, 2, 64), generator=gen).float() * factor
                v = torch.randn((T, 2, 64), generator=gen)
                q = torch.randint(-8, 9, q.shape, generator=gen).to(q_t)
                s = torch.tensor(slots, dtype=torch.int32)
                c.expect(k, v, s)
                bd.bd_kv_write(c.kv, k.to(DEV), v.to(DEV), s.to(DEV))
                out, lse = run_attend(bd, c, q, table, lens_t, scale / factor)
                out, lse, at = ref.to64(out), ref.to64(lse), 0
                for b, n in enumerate(lens):
                    kr = np.stack([c.row64(0, x) for x in slots[at:at + n]])
                    vr = np.stack([c.row64(1, x) for x in slots[at:at + n]])
                    at += n
                    want, want_lse, _ = ref.attend(ref.to64(q)[b], kr, vr, scale / factor)
                    tol = 2.0 ** -8 * np.abs(want) + (n + 64) * U * np.abs(vr).max()
                    assert np.all(np.abs(out[b] - want) <= tol), (b, np.abs(out[b] - want).max())
                    # one rounding of the product, one of the logarithm of a number of ties
                    assert np.all(np.abs(lse[b] - want_lse) <= 4 * U * np.abs(want_lse) + 16 * U)


# ----------------------------------------------------------------------------
# rows that are split and joined, by wide tables

@pytest.mark.parametrize("dim", [16, 48, 64, 80, 96, 112, 128, 144, 176, 192, 240, 256])
@pytest.mark.parametrize("kind", [BF, E4])
@pytest.mark.parametrize("q_t", [BF, F32])
def test_wide_lengths(bd, dim, kind, q_t):
    print("wide", dim, kind, q_t, flush=True)
    for heads, group, page, layout in ((2, 4, 16, "heads"), (1, 8, 24, "tokens")):
        c, q, table, lens, slots = attend_case(bd, EDGES, heads, group, dim, page, kind, q_t, layout)
        table = widened(table, page)
        assert is_split(c, q, table)
        out, lse = run_attend(bd, c, q, table, lens)
        check_attend(c, q, EDGES, slots, out, lse, dim ** -0.5)
        again, lse2 = run_attend(bd, c, q, table, lens)
        assert same_bits(out, again) and same_bits(lse, lse2)


@pytest.mark.parametrize("heads,group", [(1, 1), (3, 1), (2, 2), (1, 7), (2, 16), (1, 17), (2, 33), (1, 64), (9, 3)])
def test_wide_head_layouts(bd, heads, group):
    """Rows of one unit and of two dozen, each cut wherever it can be; more than 16 query heads to a key-value head,
    the last 16 not all there; and some of the same rows while thousands of others are there, where few are cut."""
    print("wide heads", heads, group, flush=True)
    for kind, dim, page in ((E4, 64, 8), (BF, 128, 48)):
        lens = [5, 0, 3000, 64, 200]
        c, q, table, lens_t, slots = attend_case(bd, lens, heads, group, dim, page, kind, BF, "both")
        table = widened(table, page)
        assert is_split(c, q, table)
        out, lse = run_attend(bd, c, q, table, lens_t)
        check_attend(c, q, lens, slots, out, lse, dim ** -0.5)
        pick = torch.arange(203) * 3 % 5
        many, many_lse = run_attend(bd, c, q[pick].contiguous(), table[pick].contiguous(), lens_t[pick])
        first = np.concatenate([[0], np.cumsum(lens)])
        own = [t for i in pick for t in slots[first[i]:first[i + 1]]]
        check_attend(c, q[pick], [lens[i] for i in pick], own, many, many_lse, dim ** -0.5, rows=(0, 1, 2, 4, 119, 202))


@pytest.mark.parametrize("B", [65, 513, 4099, 100003])
def test_wide_many_sequences(bd, B):
    """More sequences than a wave has lanes, most of them short: the line of units is worked out over all of them."""
    lens = [0, 1, 30, 64, 130, 7, 128, 129]
    c, q, table, lens_t, slots = attend_case(bd, lens, 1, 2, 32, 16, E4, BF)
    table = widened(table, 16)
    pick = torch.arange(B) * 5 % len(lens)
    q_all, table_all, lens_all = q[pick].contiguous(), table[pick].contiguous(), lens_t[pick].contiguous()
    bad = list(range(11, B, 97))
    lens_all[bad] = 4097
    assert is_split(c, q_all, table_all)
    out, lse = run_attend(bd, c, q_all, table_all, lens_all)
    alone, alone_lse = run_attend(bd, c, q, table, lens_t)
    check_attend(c, q, lens, slots, alone, alone_lse, 32 ** -0.5)
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    # a row may be cut elsewhere in another batch: two bf16 roundings and the sums' own
    fine = np.setdiff1d(np.arange(B), bad)
    o, a = ref.to64(out)[fine], ref.to64(alone)[pick.numpy()][fine]
    assert np.all(np.abs(o - a) <= 2.0 ** -7 * np.abs(a) + 2.0 ** -14)


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_wide_scales(bd, scale):
    for kind in (BF, E4):
        lens = [1, 40, 400]
        c, q, table, lens_t, slots = attend_case(bd, lens, 2, 2, 64, 16, kind, BF, spread=3.0)
        out, lse = run_attend(bd, c, q, widened(table, 16), lens_t, scale)
        check_attend(c, q, lens, slots, out, lse, scale)


@pytest.mark.parametrize("up", [1, -1])
@pytest.mark.parametrize("kind", [BF, E4])
def test_wide_rising_scores(bd, kind, up):
    """Scores that rise by far more than the running maximum's slack from part to part, and fall."""
    c, q, table, lens_t, slots = attend_case(bd, [600], 1, 2, 64, 16, kind, BF)
    k = torch.zeros((600, 1, 64))
    k[:, 0, 0] = up * torch.arange(600).float()
    v = torch.randn((600, 1, 64), generator=gen_of(2))
    q = torch.zeros((1, 2, 64), dtype=BF)
    q[0, 0, 0], q[0, 1, 0] = 1.0, 0.125
    s = torch.tensor(slots, dtype=torch.int32)
    c.expect(k, v, s)
    bd.bd_kv_write(c.kv, k.to(DEV), v.to(DEV), s.to(DEV))
    out, lse = run_attend(bd, c, q, widened(table, 16), lens_t, 1.0)
    check_attend(c, q, [600], slots, out, lse, 1.0)


@pytest.mark.parametrize("q_t", [BF, F32])
def test_wide_infinite_and_nan_rows(bd, q_t):
    """Infinities and NaN in some parts of a row, the others finite: the joined row is what the formula gives."""
    lens = [700, 700, 700, 700, 700, 140]
    c, q, table, lens_t, slots = attend_case(bd, lens, 1, 2, 32, 16, BF, q_t)
    table = widened(table, 16)
    assert is_split(c, q, table)
    first = np.concatenate([[0], np.cumsum(lens)])
    T = int(first[-1])
    k = torch.randn((T, 1, 32), generator=gen_of(3)).to(BF)
    v = torch.randn((T, 1, 32), generator=gen_of(4)).to(BF)
    q = q.abs() + 0.1
    inf = float("inf")
    k[first[0] + 128:first[0] + 256, 0, 0] = -inf     # a part whose scores are all -infinity
    k[first[0] + 640:first[0] + 700, 0, 1] = -inf     # the last one too
    v[first[1] + 300, 0, 3] = inf                     # an infinite value in a middle part
    k[first[2] + 650, 0, 1] = float("nan")            # NaN scores in the last part
    v[first[3] + 5, 0, 2] = float("nan")              # a NaN value in the first
    k[first[4]:first[4] + 128, 0, 5] = -inf           # the first part all -infinity
    k[first[5]:, 0, 0] = -inf                         # every score of both parts: NaN, as in the formula
    s = torch.tensor(slots, dtype=torch.int32)
    c.expect(k, v, s)
    bd.bd_kv_write(c.kv, k.to(DEV), v.to(DEV), s.to(DEV))
    out, lse = run_attend(bd, c, q, table, lens_t)
    o = ref.to64(out)
    if q_t == BF:
        check_attend(c, q, lens, slots, out, lse, 32 ** -0.5, rows=(0, 4))
    else:
        assert np.isfinite(o[[0, 4]]).all() and lse[[0, 4]].isfinite().all()
    assert np.isposinf(o[1, :, 3]).all() and np.isfinite(np.delete(o[1], 3, 1)).all()
    assert np.isnan(o[2]).all() and lse[2].isnan().all()
    assert np.isnan(o[3, :, 2]).all() and np.isfinite(np.delete(o[3], 2, 1)).all()
    assert np.isnan(o[5]).all()


def test_wide_pages_and_lengths_out_of_range(bd):
    for kind in (BF, E4):
        lens = [200, 900, 200, 30, 1000, 50]
        c, q, table, lens_t, slots = attend_case(bd, lens, 2, 2, 64, 16, kind, BF)
        bad, bad_len = widened(table, 16), lens_t.clone()
        bad[1, 56] = -1                      # the last page in use, in the last part
        bad[2, 0] = c.kv.num_pages
        bad[4, 30] = 2 ** 31 - 1             # a middle part
        bad_len[3] = -5
        bad_len[5] = 4097
        out, lse = run_attend(bd, c, q, bad, bad_len)
        for b in (1, 2, 4, 5):
            assert out[b].isnan().all() and lse[b].isnan().all()
        assert (out[3] == 0).all() and (lse[3] == -float("inf")).all()
        check_attend(c, q, lens, slots, out, lse, 0.125, rows=(0,))


def test_wide_graph(bd):
    """A captured call on a wide table, replayed while the lengths change so that rows are cut elsewhere each time, with
    eager calls of other sizes between the replays; every replay against the eager result and the formula."""
    longest = [2000, 700, 1, 300]
    for kind in (E4, BF):
        c, q, table, lens_t, slots = attend_case(bd, longest, 2, 4, 64, 16, kind, BF)
        table = widened(table, 16)
        assert is_split(c, q, table)
        gq, gt, gl = q.to(DEV), table.to(DEV), lens_t.to(DEV)
        lse = torch.empty(q.shape[:2], dtype=F32, device=DEV)
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            bd.bd_attend(gq, c.kv, gt, gl, lse=lse)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = bd.bd_attend(gq, c.kv, gt, gl, lse=lse)
        first = np.concatenate([[0], np.cumsum(longest)])
        for lens in ([2000, 700, 1, 300], [1, 1, 1, 1], [0, 0, 0, 0], [129, 700, 0, 128], [1999, 0, 1, 299],
                     [2000, 700, 1, 300]):
            gl.copy_(torch.tensor(lens))
            held.fill_(7.0)
            lse.fill_(7.0)
            graph.replay()
            got, got_lse = held.clone(), lse.clone()
            bd.bd_attend(gq[:1], c.kv, gt[:1, :8], torch.full_like(gl[:1], 100))
            torch.cuda.synchronize()
            eager, eager_lse = run_attend(bd, c, q, table, torch.tensor(lens, dtype=torch.int32))
            assert same_bits(got, eager) and same_bits(got_lse, eager_lse), lens
            own = [t for b, n in enumerate(lens) for t in slots[first[b]:first[b] + n]]
            check_attend(c, q, lens, own, got, got_lse, 0.125)


@pytest.mark.parametrize("dim", [16, 64, 96, 128, 160, 192, 256])
@pytest.mark.parametrize("kind", [BF, E4])
@pytest.mark.parametrize("wide", [False, True])
def test_fp32_queries_hold_their_bits(bd, dim, kind, wide):
    """Scores of fp32 queries in all of their 24 bits.  Every key has one value that is not 0, a power of two, so that a
    score is one query value times it, exactly, in whatever terms and order it is summed; two terms of 8 bits would be
    off by up to 2^-17 of it.  The tokens' scores differ by 0 or more than 2^7 (after scale), so lse is the largest score
    and the logarithm of how many have it: one rounding of each product and of the sum."""
    print("fp32 queries", dim, kind, wide, flush=True)
    lens, scale = [1, 130, 300], 0.75
    c, q, table, lens_t, slots = attend_case(bd, lens, 2, 3, dim, 16, kind, F32)
    table = widened(table, 16) if wide else table
    T, gen = len(slots), gen_of(dim)
    at = torch.randint(0, dim, (T, 2), generator=gen)
    k = torch.zeros((T, 2, dim)).scatter_(2, at[..., None], 1.0)
    v = torch.randn((T, 2, dim), generator=gen)
    # the values of one query: 2^10 apart, with random bits behind
    step = torch.stack([torch.randperm(dim, generator=gen) for _ in range(len(lens) * 6)]).view(len(lens), 6, dim)
    q = step.float() * 2.0 ** 10 + torch.rand(step.shape, generator=gen) * 2.0 ** 9 + 0.1
    s = torch.tensor(slots, dtype=torch.int32)
    c.expect(k, v, s)
    bd.bd_kv_write(c.kv, k.to(DEV), v.to(DEV), s.to(DEV))
    out, lse = run_attend(bd, c, q, table, lens_t, scale)
    first = 0
    for b, n in enumerate(lens):
        kr = np.stack([c.row64(0, x) for x in slots[first:first + n]])
        vr = np.stack([c.row64(1, x) for x in slots[first:first + n]])
        first += n
        want, want_lse, _ = ref.attend(ref.to64(q)[b], kr, vr, scale)
        assert np.all(np.abs(ref.to64(lse)[b] - want_lse) <= 4 * U * np.abs(want_lse) + 16 * U)
        tol = 2.0 ** -8 * np.abs(want) + (n + 64) * U * np.abs(vr).max()
        assert np.all(np.abs(ref.to64(out)[b] - want) <= tol)


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -149, 2.0 ** -140, 2.0 ** -127, -2.0 ** -126, 2.0 ** -112, -2.0 ** -110])
@pytest.mark.parametrize("wide", [False, True])
def test_small_scales_of_large_scores(bd, scale, wide):
    """Scales down to 0, of scores up to 2^119 (whole numbers up to 2^12 times 2^107, exact): a weight's exponent is off by
    the scale's own rounding, half of 2^-149 times the score at most or 2^-24 of it, and a few roundings."""
    lens = [1, 40, 300, 129]
    for q_t in (BF, F32):
        for kind in (BF, E4):
            print("small scales", scale, wide, q_t, kind, flush=True)
            c, q, table, lens_t, slots = attend_case(bd, lens, 2, 2, 64, 16, kind, q_t)
            table = widened(table, 16) if wide else table
            T, gen = len(slots), gen_of(9)
            k = torch.randint(-8, 9, (T, 2, 64), generator=gen).float() * 2.0 ** 107
            v = torch.randn((T, 2, 64), generator=gen)
            q = torch.randint(-8, 9, q.shape, generator=gen).to(q_t)
            s = torch.tensor(slots, dtype=torch.int32)
            c.expect(k, v, s)
            bd.bd_kv_write(c.kv, k.to(DEV), v.to(DEV), s.to(DEV))
            out, lse = run_attend(bd, c, q, table, lens_t, scale)
            out, lse, at = ref.to64(out), ref.to64(lse), 0
            for b, n in enumerate(lens):
                kr = np.stack([c.row64(0, x) for x in slots[at:at + n]])
                vr = np.stack([c.row64(1, x) for x in slots[at:at + n]])
                at += n
                want, want_lse, _ = ref.attend(ref.to64(q)[b], kr, vr, scale)
                score = 2.0 ** 119
                ds = 8 * U * score * abs(scale) + 2.0 ** -149 * score
                tol = 2.0 ** -8 * np.abs(want) + np.abs(vr).max() * (np.expm1(2 * ds) + 2.0 ** -15 + (n + 64) * U)
                assert np.all(np.abs(out[b] - want) <= tol), (b, np.abs(out[b] - want).max())
                assert np.all(np.abs(lse[b] - want_lse) <= ds + 4 * U * np.abs(want_lse) + (n + 64) * U)


@pytest.mark.parametrize("dim", [16, 64, 80, 96, 128, 160, 192, 224, 256])
@pytest.mark.parametrize("q_t", [BF, F32])
@pytest.mark.parametrize("wide", [False, True])
def test_infinite_keys_at_every_width(bd, dim, q_t, wide):
    """A score of -infinity drops out and an infinite value stays in its column, wherever the queries' terms are held.
    fp32 queries in a part that such a key broke are one bf16 term, half a step of it (2^-8) off."""
    print("infinite keys", dim, q_t, wide, flush=True)
    lens = [70, 300, 380]
    c, q, table, lens_t, slots = attend_case(bd, lens, 1, 3, dim, 16, BF, q_t)
    table = widened(table, 16) if wide else table[:, :24].contiguous()
    gen = gen_of(dim)
    k, v = (torch.randn((sum(lens), 1, dim), generator=gen).to(BF) for _ in range(2))
    q = (q.abs() + 0.1).to(q_t)
    k[5, 0, 0] = -float("inf")
    k[200, 0, dim - 1] = -float("inf")
    v[300, 0, 7] = float("inf")
    s = torch.tensor(slots, dtype=torch.int32)
    c.expect(k, v, s)
    bd.bd_kv_write(c.kv, k.to(DEV), v.to(DEV), s.to(DEV))
    out, lse = run_attend(bd, c, q, table, lens_t)
    out, lse, at = ref.to64(out), ref.to64(lse), 0
    for b, n in enumerate(lens):
        kr = np.stack([c.row64(0, x) for x in slots[at:at + n]])
        vr = np.stack([c.row64(1, x) for x in slots[at:at + n]])
        at += n
        want, want_lse, S = ref.attend(ref.to64(q)[b], kr, vr, dim ** -0.5)
        one_term = q_t == F32 and b < 2
        ds = (3 * dim + 8) * U * S + (2.0 ** -8 * S if one_term else 0.0)
        vmax = np.abs(vr[np.isfinite(vr)]).max()
        tol = 2.0 ** -8 * np.abs(want) + 2 * vmax * (np.expm1(2 * ds) + 2.0 ** -8 + (n + 64) * U)
        inf = np.isinf(want)
        assert np.array_equal(np.isinf(out[b]), inf) and (out[b][inf] > 0).all()
        assert np.all(np.abs(out[b][~inf] - want[~inf]) <= tol[~inf])
        assert np.all(np.abs(lse[b] - want_lse) <= ds + (n + 64) * U + 4 * U * np.abs(want_lse))
