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
