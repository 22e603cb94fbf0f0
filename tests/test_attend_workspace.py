"""The workspace of the attention of one new token: its size, and that what is split and joined stays within it."""

import pytest
import torch

import tenant_serving_amd as bd
from tenant_serving_amd import step
from tests import test_attend_formed as formed

DEV = "cuda:0"
BF, F32, E4, E2 = formed.BF, formed.F32, formed.E4, formed.E2


@pytest.mark.parametrize("dim", [80, 96, 112, 128, 192, 256])
@pytest.mark.parametrize("group", [1, 5, 8, 10, 11, 16, 17, 64])
def test_size_is_that_of_two_workgroups_per_cu(dim, group):
    """Whatever the cache's type: partial results of 512 workgroups of 16 heads in two places each, and the table."""
    for B, heads, pages in ((64, 8, 512), (1, 8, 8192), (300, 1, 512)):
        need = step._library().bd_attend_workspace_bytes(B, heads * group, heads, dim, 16, pages)
        assert 0 < need <= 512 * 2 * 16 * (dim + 2) * 4 + 16 * 768


@pytest.mark.gpu
@pytest.mark.parametrize("group", [1, 3, 10, 11, 15, 16, 17])
@pytest.mark.parametrize("kind,q_t", [(BF, BF), (E4, F32), (E2, BF)])
def test_splits_of_every_group(group, kind, q_t):
    """Long rows that many workgroups share, with the bytes that were named and not one more."""
    lens = [3000, 1, 0, 2500, 700]
    for dim in (64, 128):
        print("workspace", group, kind, dim, flush=True)
        c, q, table, n, slots = formed.case(lens, 2, group, dim, 16, kind, q_t)
        dev = [x.to(DEV) for x in (q, table, n)]
        B, pages = table.shape
        need = step._library().bd_attend_workspace_bytes(B, 2 * group, 2, dim, 16, pages)
        room = torch.full((need // 4 + 64,), 7.0, device=DEV)
        out = torch.empty(q.shape, dtype=BF, device=DEV)
        lse = torch.empty(q.shape[:2], dtype=F32, device=DEV)
        kind_q = step._IN[q.dtype]
        st = step._library().bd_attend(c.kv._ref, dev[0].data_ptr(), kind_q, step._Pair(2 * group * dim, dim), 2 * group,
                                       dev[1].data_ptr(), pages, pages, dev[2].data_ptr(), B, dim ** -0.5, out.data_ptr(),
                                       lse.data_ptr(), room.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
        assert st == 0 and need % 4 == 0
        torch.cuda.synchronize()
        assert (room[need // 4:] == 7).all()
        formed.check(c, q, slots, out, lse)
        assert formed.same_bits(out, bd.bd_attend(*(dev[0], c.kv, dev[1], dev[2])))
