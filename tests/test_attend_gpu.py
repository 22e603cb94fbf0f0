"""GPU parity of the attention of one new token where the call's form matters: page tables with far more columns than
the lengths need, as a serving program keeps them (rows are split then and joined, whatever their lengths), beside
tables just wide enough (rows stay in one piece); and scores of any size.  The plain implementation and the tolerances
are those of test_step_gpu.py unless a test derives its own."""

import numpy as np
import pytest
import torch

from tests import step_reference as ref
from tests.test_step_gpu import BF, DEV, E4, F32, U, attend_case, bd, gen_of, run_attend  # noqa: F401

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
