"""The operators of a generation together, as a server runs them: a prompt's tokens through norm, fused linears, rotary
positions, a 4-bit cache and the prompt's attention, then one token after another with the attention of one token; each
operator against its plain form on what the one before gave.  Tolerances: those of each operator's own tests."""

import numpy as np
import pytest
import torch

import tenant_serving_amd as bd
from tests import test_attend_formed as one
from tests import test_cache_four as four
from tests import test_prompt as many
from tests import test_rotary as turn
from tests.test_step_gpu import check_bf16, ref as plain

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


class Layer:
    """One attention block of a small model, its tenants' weights, and its 4-bit cache."""

    def __init__(self, seed=77, d=512, hq=8, heads=2, dim=64, page=16, tenants=3, pages=40):
        from tenant_serving_amd import synth
        self.d, self.hq, self.heads, self.dim, self.page = d, hq, heads, dim, page
        gen = synth.generator(seed, DEV)
        self.weights = {}
        for name, n in (("q", hq * dim), ("k", heads * dim), ("v", heads * dim)):
            sets = [bd.bd_compress(synth.laplace_delta(gen, n, d, 1e-3, DEV), 1) for _ in range(tenants)]
            self.weights[name] = (synth.base_weight(gen, n, d, DEV), [s for s, _ in sets], [a for _, a in sets])
        self.gain = (1 + 0.1 * torch.randn((tenants, d), generator=gen, device=DEV)).to(BF)
        self.angles = bd.bd_rotary_angles(dim, 10000.0, scaling="bands", factor=4.0, trained=256, device=DEV)
        self.c = four.Cache(pages, heads, page, dim)
        self.c.kv.k_scales.fill_(255), self.c.kv.v_scales.fill_(255)   # what is not written is NaN
        for s in self.c.scales:
            s.fill(255)

    def project(self, x, ids):
        h = bd.bd_rms_norm(x, self.gain, variant_ids=ids)
        y = [bd.bd_linear_grouped(h, ids, w, s, a, 1) for w, s, a in self.weights.values()]
        return [h] + [t.view(len(x), -1, self.dim) for t in y]

    def check_projection(self, x, ids, h, *rows):
        import oracle
        check_bf16(h, plain.rms_norm(x, self.gain, 1e-5, None, ids)[0], self.d)
        for (w, s, a), got in zip(self.weights.values(), rows):
            want = oracle.linear_grouped(h.cpu(), ids.cpu(), w.cpu(), [t.cpu().numpy() for t in s],
                                         [t.cpu().numpy() for t in a], True)
            err = plain.to64(got.reshape(len(x), -1)) - want
            assert np.linalg.norm(err) <= 1e-3 * np.linalg.norm(want)


@pytest.mark.gpu
@pytest.mark.parametrize("form", [dict(), dict(cap=8.0), dict(window=20)])
def test_prompt_then_tokens(form):
    w = Layer()
    gen = torch.Generator(device=DEV).manual_seed(5)
    chunks, tenant = [[40, 3, 33], [25, 1, 0]], [2, 0, 1]    # two chunks of three requests' prompts, one of them empty
    table = torch.randperm(40, generator=torch.Generator().manual_seed(3))[:36].view(3, 12).to(torch.int32)
    slot = lambda b, t: int(table[b, t // w.page]) * w.page + t % w.page
    window, lens = form.get("window"), [0, 0, 0]
    kw = {n: x for n, x in form.items() if n == "cap"}
    on = lambda values: torch.tensor(values, dtype=torch.int32)
    for step in range(2 + 4):
        new = chunks[step] if step < 2 else [1, 1, 1]
        place = [(b, lens[b] + i) for b, n in enumerate(new) for i in range(n)]
        lens = [a + n for a, n in zip(lens, new)]
        ids, positions = on([tenant[b] for b, _ in place]).to(DEV), on([t for _, t in place])
        slots = on([slot(b, t) for b, t in place])
        x = torch.randn((len(place), w.d), generator=gen, device=DEV)
        h, q, k, v = w.project(x, ids)
        w.check_projection(x, ids, h, q, k, v)
        tq, tk = bd.bd_rotary(w.angles, q, positions.to(DEV), k)
        v = v.to(BF)                                 # as the turned keys are
        turn.check(tq, q.cpu(), positions, w.angles)
        turn.check(tk, k.cpu(), positions, w.angles)
        w.c.expect(tk.cpu(), v.cpu(), slots)
        bd.bd_kv_write(w.c.kv, tk, v, slots.to(DEV))
        w.c.check()
        all_slots = [[slot(b, t) for t in range(n)] for b, n in enumerate(lens)]
        if step < 2:
            starts = on(np.concatenate([[0], np.cumsum(new)]))
            first = None if window is None else on([t + 1 - window for _, t in place])
            out, lse = many.run(w.c, tq, table, on(lens), starts, first=first, **kw)
            many.check(w.c, tq, starts, all_slots, out, lse, first=first, **kw)
        else:
            first = None if window is None else on([n - window for n in lens])
            out, lse = one.run(w.c, tq, table, on(lens), first=first, **kw)
            one.check(w.c, tq, all_slots, out, lse, first=first, **kw)


@pytest.mark.gpu
def test_graph_of_a_token():
    """A token's rotary, write and attention captured once and replayed while positions, slots and lengths move on, a
    prompt's chunk run eagerly between the replays; each against the same calls made eagerly on a cache of their own."""
    B, hq, heads, dim, page, most = 3, 8, 2, 128, 16, 20
    angles = bd.bd_rotary_angles(64, interleaved=True, device=DEV)
    held = [four.Cache(B * most, heads, page, dim).kv for _ in range(2)]
    for kv in held:
        kv.k_scales.fill_(127), kv.v_scales.fill_(127)
    table = torch.randperm(B * most, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(B, most)
    dev_table = table.to(DEV)
    q, k, v = (torch.zeros((B, n, dim), device=DEV) for n in (hq, heads, heads))
    positions, slots, lens = (torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(3))
    slopes = torch.exp2(-torch.arange(1, hq + 1, device=DEV).float())

    def step(kv):
        tq, tk = bd.bd_rotary(angles, q, positions, k)
        bd.bd_kv_write(kv, tk, v.to(BF), slots)
        return bd.bd_attend(tq, kv, dev_table, lens, slopes=slopes)

    slots.fill_(-1)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(held[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(held[0])
    gen = torch.Generator().manual_seed(9)
    at = lambda b, t: int(table[b, t // page]) * page + t % page
    n = [0, 40, 200]
    for i in range(6):
        add = [i % 3, 5, 0]                      # a chunk of some prompts first, eagerly
        T = sum(add)
        place = [(b, n[b] + j) for b, a in enumerate(add) for j in range(a)]
        n = [a + b for a, b in zip(n, add)]
        cq, ck, cv = (torch.randn((T, h, dim), generator=gen).to(DEV) for h in (hq, heads, heads))
        chunk = []
        for kv in held:
            tq, tk = bd.bd_rotary(angles, cq, torch.tensor([t for _, t in place], dtype=torch.int32, device=DEV), ck)
            bd.bd_kv_write(kv, tk, cv.to(BF), torch.tensor([at(*x) for x in place], dtype=torch.int32, device=DEV))
            starts = torch.tensor(np.concatenate([[0], np.cumsum(add)]), dtype=torch.int32, device=DEV)
            chunk.append(bd.bd_attend_prompt(tq, kv, dev_table, torch.tensor(n, dtype=torch.int32, device=DEV), starts))
        assert turn.same_bits(*chunk)
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=gen))
        positions.copy_(torch.tensor(n))
        slots.copy_(torch.tensor([at(b, t) for b, t in enumerate(n)]))
        n = [t + 1 for t in n]
        lens.copy_(torch.tensor(n))
        graph.replay()
        replayed = got.clone()
        assert turn.same_bits(replayed, step(held[1]))
        assert bool(replayed.isfinite().all())
        for name in ("k", "v", "k_scales", "v_scales"):
            assert torch.equal(*(getattr(kv, name).view(torch.uint8) for kv in held)), (i, name)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [BF, torch.float8_e4m3fn, torch.float4_e2m1fn_x2])
def test_nothing_to_do(kind):
    """No tokens, no sequences, sequences without tokens, and a cache of one page with bad tables: zeros, or no rows."""
    on = lambda *values: torch.tensor(values, dtype=torch.int32, device=DEV)
    kv = bd.bd_kv_cache.empty(1, 2, 8, 64, kind, DEV)
    angles = bd.bd_rotary_angles(64, device=DEV)
    q, k = torch.ones((3, 4, 64), dtype=BF, device=DEV), torch.ones((3, 2, 64), dtype=BF, device=DEV)
    none = on()
    tq, tk = bd.bd_rotary(angles, q[:0], none, k[:0])
    assert tq.shape == (0, 4, 64) and tk.shape == (0, 2, 64)
    bd.bd_kv_write(kv, k[:0], k[:0], none)
    assert bd.bd_kv_read(kv, none)[0].shape == (0, 2, 64)
    table = torch.full((2, 5), -1, dtype=torch.int32, device=DEV)
    assert bd.bd_attend(q[:0], kv, table[:0], none, cap=3.0).shape == (0, 4, 64)
    assert bd.bd_attend_prompt(q[:0], kv, table, on(0, 0), on(0, 0, 0)).shape == (0, 4, 64)
    out = torch.full((3, 4, 64), 5.0, dtype=BF, device=DEV)
    assert bool((bd.bd_attend_prompt(q, kv, table[:0], none, on(0), out=out) == 5).all())
    for lens in (on(0, 0), on(-3, 0)):
        for kw in (dict(), dict(cap=3.0)):
            assert bool((bd.bd_attend(q[:2], kv, table, lens, **kw) == 0).all())
            out.fill_(5.0)
            bd.bd_attend_prompt(q, kv, table, lens, on(0, 2, 2), out=out, **kw)
            assert bool((out[:2] == 0).all()) and bool((out[2:] == 5).all())
    # a window that has passed the sequence's end, and one key that everything sees
    assert bool((bd.bd_attend(q[:2], kv, table, on(1, 40), first=on(1, 40)) == 0).all())
    bd.bd_kv_write(kv, k[:1], k[:1], on(0))
    table[0, 0] = 0
    for n in (1, 2, 3):
        first, last = torch.zeros(n, dtype=torch.int32, device=DEV), torch.ones(n, dtype=torch.int32, device=DEV)
        got = bd.bd_attend_prompt(q[:n], kv, table[:1], on(n), on(0, n), first=first, last=last)
        assert bool((got == 1).all())
    assert bool((bd.bd_attend(q[:1], kv, table[:1], on(1)) == 1).all())
