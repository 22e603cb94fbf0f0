"""Refusals of the rotary call, by the C ABI and by the binding, the angles' numbers, and GPU parity against the plain
64-bit form of tests/more_reference.py.

Tolerance: sine and cosine are off by at most 4 u (u = 2^-24: the angle's conversion, the series' last sums, the gain),
each product and sum by one more, so a result is off by 8 u times the sum of its two terms' magnitudes, and a bf16 one by
half a step, 2^-8 of itself, besides."""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import tenant_serving_amd as bd
from tenant_serving_amd import rotary, step
from tests import more_reference as ref

DEV = "cuda:0"
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
FAKE = 1 << 20
OFF = FAKE + 2
OK, NULL, SHAPE, ALIGN, MODE = 0, 1, 2, 3, 5


def gen_of(seed):
    return torch.Generator().manual_seed(seed)


def same_bits(a, b):
    a, b = a.detach().cpu().contiguous(), b.detach().cpu().contiguous()
    return a.dtype == b.dtype and a.shape == b.shape and torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ----------------------------------------------------------------------------
# refusals and the angles, on the host

def test_c_refusals():
    lib = step._library()

    def call(rows=({},), **c):
        base = dict(x=FAKE, out=FAKE, xs=(256, 64), os=(256, 64), heads=4)
        table = (rotary._RotaryRows * 2)()
        for i, change in enumerate(rows):
            r = {**base, **change}
            table[i] = rotary._RotaryRows(r["x"], r["out"], step._Pair(*r["xs"]), step._Pair(*r["os"]), r["heads"])
        a = dict(rows=table, count=len(rows), x_type=0, out_type=0, dim=64, turned=32, inter=0, positions=FAKE,
                 steps=FAKE, gain=1.0, T=3, stream=None)
        a.update(c)
        return lib.bd_rotary(*a.values())

    for change, want in [(dict(rows=None), NULL), (dict(positions=None), NULL), (dict(steps=None), NULL),
                         (dict(x_type=2), MODE), (dict(out_type=2), MODE), (dict(out_type=4), MODE),
                         (dict(count=0), SHAPE), (dict(count=3), SHAPE), (dict(dim=0), SHAPE), (dict(dim=72), SHAPE),
                         (dict(dim=272), SHAPE), (dict(turned=0), SHAPE), (dict(turned=31), SHAPE),
                         (dict(turned=66), SHAPE), (dict(turned=-2), SHAPE), (dict(gain=float("inf")), SHAPE),
                         (dict(gain=float("nan")), SHAPE), (dict(T=-1), SHAPE), (dict(T=1 << 31), SHAPE),
                         (dict(positions=OFF), ALIGN), (dict(steps=FAKE + 4), ALIGN)]:
        if "rows" in change:
            assert lib.bd_rotary(None, 1, 0, 0, 64, 32, 0, FAKE, FAKE, 1.0, 3, None) == want
        else:
            assert call(**change) == want, change
    for change, want in [(dict(x=None), NULL), (dict(out=None), NULL), (dict(heads=0), SHAPE), (dict(heads=65536), SHAPE),
                         (dict(xs=(-8, 64)), SHAPE), (dict(xs=(260, 64)), ALIGN), (dict(os=(256, 68)), ALIGN),
                         (dict(os=(256, -64)), SHAPE), (dict(x=OFF), ALIGN), (dict(out=OFF), ALIGN)]:
        assert call(rows=({}, change)) == want, change
        assert call(rows=(change,)) == want, change
    assert call(rows=(dict(x=None, out=None),), T=0, positions=None) == OK


def test_binding_refusals(monkeypatch):
    a = bd.bd_rotary_angles(64, device="cpu")
    q, k, pos = torch.zeros(5, 4, 64), torch.zeros(5, 2, 64), torch.zeros(5, dtype=torch.int32)
    wide = torch.zeros(5, 10 * 64)
    wq, wk = wide[:, :256].view(5, 4, 64), wide[:, 256:384].view(5, 2, 64)
    for err, match, args, kw in [
            (TypeError, "angles", (None, q, pos), {}), (TypeError, "q must be", (a, None, pos), {}),
            (TypeError, "q must be", (a, q.double(), pos), {}), (ValueError, "head_dim", (a, torch.zeros(5, 4, 72), pos), {}),
            (ValueError, "head_dim", (a, torch.zeros(5, 256), pos), {}),
            (ValueError, "turn 64 columns", (a, torch.zeros(5, 4, 48), pos), {}),
            (ValueError, "one dtype", (a, q, pos, k.to(BF)), {}), (ValueError, "one dtype", (a, q, pos, k[:4]), {}),
            (ValueError, "k must be", (a, q, pos, torch.zeros(5, 2, 80)), {}),
            (ValueError, "k_out needs k", (a, q, pos), dict(k_out=k)),
            (TypeError, "positions", (a, q, pos.long()), {}), (ValueError, "positions", (a, q, pos[:4]), {}),
            (TypeError, "results are", (a, q, pos), dict(dtype=torch.float16)),
            (TypeError, "results are", (a, q, pos), dict(q_out=q.double())),
            (ValueError, "k_out must be", (a, q, pos, k), dict(q_out=q.to(BF), k_out=k.clone())),
            (ValueError, "q_out must be", (a, q, pos), dict(q_out=torch.zeros(5, 3, 64))),
            (ValueError, "16 bytes", (a, torch.zeros(5 * 256 + 4)[1:1281].view(5, 4, 64), pos), {}),
            (ValueError, "q_out overlaps q", (a, q[:4], pos[:4]), dict(q_out=q[1:])),
            (ValueError, "q_out overlaps k", (a, q[:, :2], pos, k), dict(q_out=k)),
            (ValueError, "q_out overlaps k", (a, wq, pos, wk), dict(q_out=wide[:, 320:576].view(5, 4, 64))),
            (ValueError, "q_out overlaps k_out", (a, q, pos, k), dict(q_out=wq, k_out=wide[:, 192:320].view(5, 2, 64))),
            (ValueError, "overlap", (a, q, pos), dict(q_out=torch.zeros(1, 4, 64).expand(5, 4, 64))),
            (ValueError, "q_out overlaps positions", (a, q[:, :1], q.view(torch.int32)[0, 0, :5]),
             dict(q_out=torch.as_strided(q, (5, 1, 64), (256, 64, 1)))),
            (ValueError, "GPU", (a, q, pos), {}), (ValueError, "GPU", (a, wq, pos, wk), dict(q_out=wq, k_out=wk)),
            (ValueError, "GPU", (a, wq, pos, wk), dict(k_out=wk))]:
        with pytest.raises(err, match=match):
            bd.bd_rotary(*args, **kw)
    with pytest.raises(ValueError, match="q_out overlaps the angles"):
        bd.bd_rotary(a, q[:1, :1], pos[:1], q_out=a.steps.view(F32).view(1, 1, 64))


def test_rows_apart():
    wide = torch.zeros(6, 9, 32)
    for a, b, want in [(wide[:, :4], wide[:, 4:6], True), (wide[:, :4], wide[:, 3:6], False),
                       (wide[:, 0:9:2], wide[:, 1:9:2], True), (wide[:, 0:9:2], wide[:, 2:4], False),
                       (wide[:3], wide[3:], True), (wide[:4], wide[3:], False), (wide[0::2], wide[1::2], True),
                       (wide[0::2, :2], wide[1:3, 1:2], False), (wide[:, :, :16], wide[:, :, 16:], True),
                       (wide[:1], wide[:1, 8:], False), (wide[:1, :8], wide[:1, 8:], True)]:
        assert rotary._rows_apart(a, b) is want and rotary._rows_apart(b, a) is want


def test_angles():
    pi = Fraction(math.pi)
    for kw, f in [({}, lambda i: 10000.0 ** (-i / 16)), (dict(scaling="linear", factor=4.0), lambda i: 10000.0 ** (-i / 16) / 4),
                  (dict(scaling="base", factor=8.0), lambda i: (10000.0 * 8.0 ** (32 / 30)) ** (-i / 16))]:
        a = bd.bd_rotary_angles(32, 10000.0, device="cpu", **kw)
        for i, s in enumerate(a.steps.tolist()):
            want = Fraction(f(i)) / (2 * pi) * 2 ** 64
            assert abs((s % 2 ** 64) - want) <= 2 ** 12     # a float64's accuracy
    a = bd.bd_rotary_angles(64, 1e6, scaling="bands", factor=8.0, trained=4096, low=1.0, high=32.0, device="cpu")
    for i, x in enumerate(a.frequencies):
        f = 1e6 ** (-i / 32)
        turns = 4096 * f / (2 * math.pi)
        assert f / 8 * (1 - 1e-12) <= x <= f * (1 + 1e-12)
        assert (turns < 32 or x == f) and (turns > 1 or x == f / 8)
    assert a.frequencies == sorted(a.frequencies, reverse=True)
    b = bd.bd_rotary_angles(64, frequencies=torch.tensor(a.frequencies, dtype=torch.float64), device="cpu")
    assert torch.equal(a.steps, b.steps)
    for err, kw in [(ValueError, dict(turned=3)), (ValueError, dict(turned=0)), (ValueError, dict(turned=258)),
                    (ValueError, dict(turned=8, base=0.0)), (ValueError, dict(turned=8, factor=-1.0, scaling="linear")),
                    (ValueError, dict(turned=8, scaling="other")), (ValueError, dict(turned=8, scaling="bands")),
                    (ValueError, dict(turned=2, scaling="base", factor=2.0)), (ValueError, dict(turned=8, gain=math.nan)),
                    (ValueError, dict(turned=8, frequencies=[1.0])),
                    (ValueError, dict(turned=2, frequencies=[math.inf]))]:
        with pytest.raises(err):
            bd.bd_rotary_angles(device="cpu", **kw)


# ----------------------------------------------------------------------------
# on the GPU

def check(got, x, positions, angles):
    want, size = ref.rotary(x.double().numpy(), positions.numpy(), angles.frequencies, angles.turned, angles.interleaved,
                            angles.gain)
    got64 = got.cpu().double().numpy()
    assert np.array_equal(np.isfinite(got64), np.isfinite(want))
    tol = 8 * U * size + (2.0 ** -8 * np.abs(want) if got.dtype == BF else 0.0) + 2.0 ** -133
    with np.errstate(invalid="ignore"):
        off = ~(np.abs(got64 - want) <= tol) & np.isfinite(want)
    assert not off.any(), np.argwhere(off)[:4].tolist()
    if angles.turned < x.shape[2]:      # the others are copies, rounded once where the type is narrower
        assert same_bits(got.cpu()[..., angles.turned:], x[..., angles.turned:].to(got.dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("dim,turned", [(16, 2), (16, 16), (64, 64), (64, 16), (80, 20), (80, 80), (96, 24), (112, 6),
                                        (128, 128), (128, 64), (192, 48), (256, 256), (256, 250)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_sizes(dim, turned, interleaved):
    print("rotary", dim, turned, interleaved, flush=True)
    angles = bd.bd_rotary_angles(turned, 500000.0, interleaved=interleaved, gain=1.25, device=DEV)
    for T, heads, k_heads in ((1, 1, 1), (3, 9, 2), (67, 5, 5), (700, 8, 1)):
        gen = gen_of(T)
        pos = torch.randint(-70000, 1 << 20, (T,), generator=gen, dtype=torch.int32)
        for x_t, o_t in ((F32, BF), (BF, BF), (BF, F32), (F32, F32)):
            q = torch.randn((T, heads, dim), generator=gen).to(x_t)
            k = torch.randn((T, k_heads, dim), generator=gen).to(x_t)
            gq, gk = bd.bd_rotary(angles, q.to(DEV), pos.to(DEV), k.to(DEV), dtype=o_t)
            assert gq.dtype == gk.dtype == o_t
            check(gq, q, pos, angles)
            check(gk, k, pos, angles)
            assert same_bits(bd.bd_rotary(angles, q.to(DEV), pos.to(DEV), dtype=o_t), gq)


@pytest.mark.gpu
def test_positions_far_and_back():
    """Every position an int32 has, and back by its negative."""
    angles = bd.bd_rotary_angles(64, 1e4, device=DEV)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31 + 1, -2 ** 31, 123456789, 65536, -65537], dtype=torch.int32)
    x = torch.randn((9, 3, 64), generator=gen_of(1))
    y = bd.bd_rotary(angles, x.to(DEV), pos.to(DEV), dtype=F32)
    # float64's product of a position and a frequency is off by 2^-53 of up to 2^31: 2^-22, and its reduction alike
    want, size = ref.rotary(x.double().numpy(), pos.numpy(), angles.frequencies, 64, False)
    assert np.all(np.abs(y.cpu().double().numpy() - want) <= (8 * U + 2.0 ** -21) * size)
    assert same_bits(y[0], x[0])
    back = bd.bd_rotary(angles, y[:5], -pos.to(DEV)[:5], dtype=F32)
    assert np.all(np.abs(back.cpu().double().numpy() - x[:5].double().numpy()) <= 32 * U * size[:5])


@pytest.mark.gpu
def test_methods_of_scaling():
    gen = gen_of(4)
    pos = torch.randint(0, 1 << 17, (50,), generator=gen, dtype=torch.int32)
    x = torch.randn((50, 2, 128), generator=gen)
    for kw in (dict(scaling="linear", factor=16.0), dict(scaling="base", factor=16.0),
               dict(scaling="bands", factor=16.0, trained=8192), dict(scaling="bands", factor=8.0, trained=4096, low=1.0, high=32.0, gain=1.2)):
        angles = bd.bd_rotary_angles(128, 500000.0, device=DEV, **kw)
        check(bd.bd_rotary(angles, x.to(DEV), pos.to(DEV)), x, pos, angles)


@pytest.mark.gpu
@pytest.mark.parametrize("x_t", [F32, BF])
def test_views_and_in_place(x_t):
    """Queries and keys as views of one q, k, v result, turned in place or into other views; nothing else changes."""
    T, hq, h, dim = 33, 6, 2, 96
    angles = bd.bd_rotary_angles(32, 1e4, device=DEV)
    gen = gen_of(5)
    qkv = torch.randn((T, (hq + 2 * h) * dim + 16), generator=gen).to(x_t)
    pos = torch.arange(T, dtype=torch.int32)
    views = lambda t: (t[:, :hq * dim].view(T, hq, dim), t[:, hq * dim:(hq + h) * dim].view(T, h, dim))  # noqa: E731
    q, k = views(qkv)
    dev = qkv.to(DEV)
    dq, dk = views(dev)
    want = bd.bd_rotary(angles, dq, pos.to(DEV), dk, dtype=x_t)
    check(want[0], q, pos, angles)
    check(want[1], k, pos, angles)
    got = bd.bd_rotary(angles, dq, pos.to(DEV), dk, q_out=dq, k_out=dk)
    assert got[0] is dq and same_bits(dq, want[0]) and same_bits(dk, want[1])
    assert same_bits(dev[:, (hq + h) * dim:], qkv[:, (hq + h) * dim:])
    # heads outermost, and one of the two allocated
    dev = qkv.to(DEV)
    dq, dk = views(dev)
    to = torch.full((hq, T + 1, dim), 7.0, dtype=x_t, device=DEV)
    a, b = bd.bd_rotary(angles, dq, pos.to(DEV), dk, q_out=to[:, :T].transpose(0, 1))
    assert same_bits(a, want[0]) and same_bits(b, want[1]) and b.dtype == x_t and (to[:, T] == 7).all()
    assert same_bits(dev, qkv)


@pytest.mark.gpu
def test_infinities_stay_in_their_pairs():
    angles = bd.bd_rotary_angles(32, 1e4, interleaved=True, device=DEV)
    x = torch.randn((4, 1, 64), generator=gen_of(2))
    x[1, 0, 5], x[2, 0, 40], x[3, 0, 0] = math.inf, -math.inf, math.nan
    pos = torch.tensor([3, 4, 5, 6], dtype=torch.int32)
    y = bd.bd_rotary(angles, x.to(DEV), pos.to(DEV), dtype=F32).cpu()
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[1, 0, 4:6], want[2, 0, 40], want[3, 0, 0:2] = True, True, True
    assert torch.equal(bad, want) and y[2, 0, 40] == -math.inf


@pytest.mark.gpu
def test_many_tokens_and_heads():
    angles = bd.bd_rotary_angles(16, 1e4, device=DEV)
    for T, hq, h in ((70001, 3, 1), (2, 65535, 7), (5, 100, 1000)):
        gen = gen_of(T)
        q, k = torch.randn((T, hq, 16), generator=gen), torch.randn((T, h, 16), generator=gen)
        pos = torch.randint(0, 9999, (T,), generator=gen, dtype=torch.int32)
        a, b = bd.bd_rotary(angles, q.to(DEV), pos.to(DEV), k.to(DEV))
        check(a, q, pos, angles)
        check(b, k, pos, angles)
    none = torch.empty((0, 2, 16), device=DEV)
    assert bd.bd_rotary(angles, none, pos[:0].to(DEV)).shape == (0, 2, 16)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Rows past 4 GiB of their tensors."""
    angles = bd.bd_rotary_angles(128, 1e4, device=DEV)
    T, step_ = 5, 1 << 29
    base = torch.empty(4 * step_ + 256, dtype=BF, device=DEV)
    q = torch.as_strided(base, (T, 2, 128), (step_, 128, 1))
    x = torch.randn((T, 2, 128), generator=gen_of(3)).to(BF)
    q.copy_(x.to(DEV))
    pos = torch.arange(T, dtype=torch.int32) * 1000
    check(bd.bd_rotary(angles, q, pos.to(DEV)), x, pos, angles)
    bd.bd_rotary(angles, q, pos.to(DEV), q_out=q)
    check(q, x, pos, angles)


@pytest.mark.gpu
def test_streams_graphs_and_devices(monkeypatch):
    angles = bd.bd_rotary_angles(64, 1e4, device=DEV)
    gen = gen_of(9)
    q = torch.randn((40, 8, 64), generator=gen).to(DEV)
    pos = torch.randint(0, 1000, (40,), generator=gen, dtype=torch.int32).to(DEV)
    want = bd.bd_rotary(angles, q, pos)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for _ in range(5):
            got = bd.bd_rotary(angles, q, pos)
    s.synchronize()
    assert same_bits(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = bd.bd_rotary(angles, q, pos)
    for i in range(3):
        q.copy_(torch.randn((40, 8, 64), generator=gen))
        pos.add_(i)
        graph.replay()
        torch.cuda.synchronize()
        assert same_bits(held, bd.bd_rotary(angles, q, pos))
    real, left = step._current_device, [1]
    monkeypatch.setattr(step, "_current_device", lambda: left.pop() if left else real())
    assert same_bits(bd.bd_rotary(angles, q, pos), held) and not left
