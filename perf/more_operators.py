"""What is measured of the operators that a request's prompt and a longer generation need next to the norm, the
8-bit cache and the attention of one new token: rotary positions, a cache held in 4 bits with the attention that
reads it, scores that are capped, biased or masked, and the attention of a prompt's tokens.

A case is a dict of plain values; `prepare` makes its inputs, `run` makes one pass: in elementary torch
operations where `own` is false, through the package's entry points where it is true.  `exact` has the same
results in 64 bits from the operators' definitions.

The definitions, in short:

  rotary  a pair (a, b) of the first r columns of a row at position p becomes g (a cos t - b sin t, b cos t + a sin t),
          t = p f: pair i is (i, i + r/2) or (2i, 2i + 1), f = base^(-2i/r), scaled for long contexts by a method
  cache   rows of keys and values go to their slots of a paged cache as e2m1 codes (4 bits) with one power-of-two
          scale per 32 columns, and are read back as bf16 (codes times scale, exactly)
  attend  softmax(s) v of one new token per sequence over the pages of its table; s = scale q k^T, or
          cap tanh(scale q k^T / cap) - slope |p - j| of its head, over the keys j in [first, length)
  prompt  the same for several new tokens of each sequence, which are its last ones: token at position p sees the
          keys j in [first, last), where nothing else is said those up to its own

The scale of a group of e2m1 codes is 2^e with the smallest e for which its largest magnitude is at most 6 * 2^e
(e no lower than -125), stored as the byte e + 127; that of a row of e4m3 codes likewise with 448 (e4m3 caches are
inputs here, not written).
"""
import math

import torch

own = False

DEV = "cuda"
BASE = 500000.0
TRAINED = 8192  # tokens of the context that the scaled frequencies are stretched from


# ----------------------------------------------------------------------------
# cases

def listed():
    return [
        # the 16 new tokens of a decode step deep in a stretched context, half of each head turned; latency
        dict(name="rotary one step", op="rotary", tokens=16, q_heads=64, heads=8, dim=128, turned=64, interleaved=True, scaling="bands", far=131072, x="float32"),
        # a long prompt's queries and keys from the fp32 results of their projections
        dict(name="rotary long prompt", op="rotary", tokens=16384, q_heads=64, heads=8, dim=128, turned=128, interleaved=False, scaling="bands", far=16384, x="float32"),
        # the new tokens of a decode step go into a 4-bit cache and are read back
        dict(name="cache decode 4 bits", op="cache", tokens=16, heads=8, dim=128, page=16, x="bfloat16"),
        # a long prompt quantised into the cache and read back
        dict(name="cache prompt 4 bits", op="cache", tokens=16384, heads=8, dim=128, page=32, x="float32"),
        # 64 ragged requests on a 4-bit cache
        dict(name="attend batch 4 bits", op="attend", batch=64, longest=16381, q_heads=64, heads=8, dim=128, page=32, q="bfloat16", kind="e2m1", cap=0.0, slopes=False, window=0),
        # one long context in 4 bits, where only a split over its length fills the GPU
        dict(name="attend one long 4 bits", op="attend", batch=1, longest=131071, q_heads=64, heads=8, dim=128, page=16, q="bfloat16", kind="e2m1", cap=0.0, slopes=False, window=0),
        # a layer with capped scores and a window of its last 1024 tokens
        dict(name="attend capped window", op="attend", batch=31, longest=4099, q_heads=32, heads=8, dim=128, page=16, q="float32", kind="bfloat16", cap=50.0, slopes=False, window=1024),
        # a bias by distance, a key-value head per query head, a small head, an 8-bit cache
        dict(name="attend distance", op="attend", batch=16, longest=8191, q_heads=32, heads=32, dim=64, page=24, q="bfloat16", kind="e4m3", cap=0.0, slopes=True, window=0),
        # five proposed tokens of each request to be checked in one pass, behind long contexts
        dict(name="prompt few tokens", op="prompt", batch=3, new=5, past=16000, q_heads=64, heads=8, dim=128, page=16, kind="bfloat16", form="causal", cap=0.0, slopes=False),
        # a chunk of a long prompt behind what a 4-bit cache holds of it
        dict(name="prompt chunk 4 bits", op="prompt", batch=1, new=512, past=32768, q_heads=64, heads=8, dim=128, page=32, kind="e2m1", form="causal", cap=0.0, slopes=False),
        # ragged prompts of several documents each, capped scores, an 8-bit cache
        dict(name="prompt documents", op="prompt", batch=7, new=2049, past=0, q_heads=32, heads=8, dim=128, page=16, kind="e4m3", form="documents", cap=30.0, slopes=False),
        # a whole prompt at once: the largest
        dict(name="prompt whole", op="prompt", batch=1, new=8192, past=0, q_heads=64, heads=8, dim=128, page=16, kind="bfloat16", form="causal", cap=0.0, slopes=False),
    ]


def _log(rng, lo, hi):
    hi = max(lo, hi)
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _kind_dim(rng):
    kind = rng.choice(["bfloat16", "e4m3", "e2m1"])
    return kind, rng.choice([64, 96, 128, 160, 192, 256] if kind == "e2m1" else [64, 80, 96, 128, 192, 256])


def draw(rng):
    op = rng.choice(["rotary", "rotary", "cache", "attend", "attend", "attend", "prompt", "prompt", "prompt"])
    heads, page = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([8, 16, 24, 32, 64, 128])
    group = rng.choice([1, 3, 4, 5, 8, 16])
    if op == "rotary":
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        turned = rng.choice([dim, dim, dim // 2, dim // 4 // 2 * 2])
        most = 16384 * 72 * 128 // (heads * (group + 1) * dim)
        return dict(op=op, tokens=_log(rng, 1, min(16384, most)), q_heads=heads * group, heads=heads, dim=dim, turned=turned, interleaved=rng.choice([False, True]), scaling=rng.choice(["none", "linear", "base", "bands"]), far=_log(rng, 64, 1 << 20), x=rng.choice(["float32", "bfloat16"]))
    if op == "cache":
        dim = rng.choice([64, 96, 128, 160, 192, 256])
        return dict(op=op, tokens=_log(rng, 1, min(16384, 16384 * 1024 // (heads * dim))), heads=heads, dim=dim, page=page, x=rng.choice(["float32", "bfloat16"]))
    kind, dim = _kind_dim(rng)
    cap, slopes = rng.choice([0.0, 0.0, 20.0, 50.0]), rng.choice([False, False, True])
    if op == "attend":
        batch = _log(rng, 1, 128)
        longest = _log(rng, 1, min(131071, 500 * 1024 * 1024 // (batch * heads * dim)))
        if kind != "e2m1" and not slopes:
            cap = cap or 30.0
        return dict(op=op, batch=batch, longest=longest, q_heads=heads * group, heads=heads, dim=dim, page=page, q=rng.choice(["float32", "bfloat16"]), kind=kind, cap=cap, slopes=slopes, window=rng.choice([0, 0, 100, 1024]))
    room = 8192 * 8192 * 64 * 128 // (heads * group * max(dim, 128)) // 4  # pairs of a query and a key
    batch = _log(rng, 1, 32)
    new = _log(rng, 1, min(8192, int(math.sqrt(room / batch)), 8192 * 64 * 128 // (batch * heads * group * dim)))
    past = rng.choice([0, _log(rng, 1, min(65536, room // batch // new, 500 * 1024 * 1024 // (batch * heads * dim)))])
    return dict(op=op, batch=batch, new=new, past=past, q_heads=heads * group, heads=heads, dim=dim, page=page, kind=kind, form=rng.choice(["causal", "causal", "window", "documents", "prefix"]), cap=cap, slopes=slopes)


def _spread(n, m):
    """n ragged numbers up to m, the same for every seed."""
    return [max(1, round(m * (1.0 - (b * 0.6180339887498949) % 1.0))) for b in range(n)]


def _lengths(c):
    """(new tokens, tokens in the cache with them) of each sequence; in a batch of more than 8 one has none."""
    n = c["batch"]
    if c["op"] == "attend":
        lens = _spread(n, c["longest"])
        new = [1] * n
    else:
        new = _spread(n, c["new"])
        past = _spread(n, c["past"])[::-1] if c["past"] else [0] * n
        lens = [a + b for a, b in zip(new, past)]
    if n > 8:
        lens[n // 2] = 0
        new[n // 2] = 1 if c["op"] == "attend" else 0
    return new, lens


def _ranges(c):
    """Per sequence the (first, last) lists of its new tokens: which keys each sees."""
    out = []
    for b, (n, length) in enumerate(zip(*_lengths(c))):
        at = list(range(length - n, length))
        first, last = [0] * n, [p + 1 for p in at]
        if c["op"] == "attend":
            first = [max(0, length - c["window"]) if c["window"] else 0]
            last = [length]
        elif c["form"] == "window":
            first = [max(0, p - 255) for p in at]
        elif c["form"] == "documents":
            size = 1 + length // (3 + b % 3)  # three to five documents
            first = [p // size * size for p in at]
        elif c["form"] == "prefix":
            upto = 1 + length * 2 // 5  # tokens that see each other in both directions
            last = [max(p + 1, upto) for p in at]
        out.append((first, last))
    return out


def _row_bytes(kind, dim):
    return {"float32": 4 * dim, "bfloat16": 2 * dim, "e4m3": dim + 1, "e2m1": dim // 2 + dim // 32}[kind]


def work(c):
    if c["op"] == "rotary":
        t, row = c["tokens"], (c["q_heads"] + c["heads"]) * c["dim"]
        turned = (c["q_heads"] + c["heads"]) * c["turned"]
        return {"bytes": t * (_row_bytes(c["x"], row) + 2 * row + 4), "flops": 3 * t * turned}
    if c["op"] == "cache":
        t, row = c["tokens"], c["heads"] * c["dim"]
        return {"bytes": t * (2 * _row_bytes(c["x"], row) + 4 * c["heads"] * _row_bytes("e2m1", c["dim"]) + 4 * row + 4), "flops": 4 * t * row}
    new, lens = _lengths(c)
    pairs = rows = pages = 0
    for first, last in _ranges(c):
        pairs += sum(max(0, b - a) for a, b in zip(first, last))
        if first and max(last) > min(first):
            rows += max(last) - min(first)
            pages += -(-max(last) // c["page"]) - min(first) // c["page"]
    values = sum(new) * c["q_heads"] * c["dim"]
    q = _row_bytes(c["q"], 1) if c["op"] == "attend" else 2
    return {"bytes": rows * 2 * c["heads"] * _row_bytes(c["kind"], c["dim"]) + values * (q + 2) + 4 * (pages + sum(new)), "flops": 4 * pairs * c["q_heads"] * c["dim"]}


# ----------------------------------------------------------------------------
# inputs

def _dtype(name):
    return {"float32": torch.float32, "bfloat16": torch.bfloat16}[name]


def _power(e):
    """2^(e - 127) from the byte."""
    return (e.to(torch.int32) << 23).view(torch.float32)


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _pack(codes):
    """Codes 0..15 along the last axis, two to a byte, the first in the low half."""
    return codes[..., 0::2] | codes[..., 1::2] << 4


def _held4(packed, exponents):
    """The fp32 values of packed codes [..., dim / 2] with scale bytes [..., dim / 32]."""
    table = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device=packed.device)
    codes = torch.stack((packed & 15, packed >> 4), -1).flatten(-2)
    x = table[codes.int()].unflatten(-1, (-1, 32))
    return (x * _power(exponents).unsqueeze(-1)).flatten(-2)


def _quantise4(x):
    """fp32 [..., dim] -> (packed codes [..., dim / 2], scale bytes [..., dim / 32])."""
    groups = x.unflatten(-1, (-1, 32))
    bits = groups.abs().amax(-1).view(torch.int32)
    e = (((bits + 0x3FFFFF) >> 23) - 2).clamp(2, 253)
    y = groups * _power(254 - e).unsqueeze(-1)
    m = y.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    m = torch.round(m / step) * step
    code = sum((m >= t).int() for t in _E2M1[1:]) | (y.view(torch.int32) < 0).int() << 3
    return _pack(code.to(torch.uint8).flatten(-2)), e.to(torch.uint8)


def _rows(gen, *shape):
    """Key, value or query rows: normal, with some channels several times as large, as projections give them."""
    loud = 1 + 4 * (torch.rand(shape[-1], generator=gen, device=DEV) > 0.95)
    return torch.randn(shape, generator=gen, device=DEV) * loud


def _cache(c, gen, pages):
    """A cache in use: every page holds rows.  Arrays [pages, heads, page, ...]; the scale bytes of e2m1 rows are
    [pages, heads, groups, page]."""
    shape = (pages, c["heads"], c["page"], c["dim"])
    got = dict(k_exp=None, v_exp=None)
    for name in ("k", "v"):
        if c["kind"] == "bfloat16":
            got[name] = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)
        elif c["kind"] == "e4m3":
            # codes of a normal row scaled to its largest value: |code| up to 448, and scales near 2^-7
            codes = torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16).mul_(110.0).clamp_(-448.0, 448.0)
            got[name] = codes.to(torch.float8_e4m3fn)
            got[name + "_exp"] = torch.randint(119, 122, shape[:3], generator=gen, device=DEV, dtype=torch.uint8)
        else:
            # codes of normal rows whose groups reach about 2.5 deviations, by lot from 4096 quantiles; scales near 2^-1
            normal = torch.special.ndtri((torch.arange(4096, device=DEV).double() + 0.5) / 4096).float() * 2
            m = normal.abs().clamp(max=6)
            codes = (torch.bucketize(m, torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)) | (normal < 0).long() << 3).to(torch.uint8)
            lot = torch.randint(0, 4096, shape[:3] + (c["dim"],), generator=gen, device=DEV, dtype=torch.int16)
            got[name] = torch.empty(shape[:3] + (c["dim"] // 2,), dtype=torch.uint8, device=DEV)
            for some in range(0, pages, 1024):
                got[name][some:some + 1024] = _pack(codes[lot[some:some + 1024].int()])
            got[name + "_exp"] = torch.randint(125, 128, (pages, c["heads"], c["dim"] // 32, c["page"]), generator=gen, device=DEV, dtype=torch.uint8)
    return got


def _handle(c, cache):
    """The package's handle of a cache, which a serving program makes once; the arrays stay the caller's."""
    if not own:
        return None
    import tenant_serving_amd as bd
    k, v = cache["k"], cache["v"]
    if c["kind"] == "e2m1":
        k, v = k.view(torch.float4_e2m1fn_x2), v.view(torch.float4_e2m1fn_x2)
    return bd.bd_kv_cache(k, v, cache["k_exp"], cache["v_exp"])


def _frequencies(c):
    """Radians per position of each pair, in float64, by the case's method of scaling to 16 times the trained context
    (the stretched bands: turns that come round more than 4 times within it stay, fewer than once are stretched)."""
    r = c["turned"]
    base = BASE * 16.0 ** (r / (r - 2)) if c["scaling"] == "base" else BASE
    f = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if c["scaling"] == "linear":
        f = [x / 16.0 for x in f]
    if c["scaling"] == "bands":
        keep = [min(1.0, max(0.0, (TRAINED * x / (2.0 * math.pi) - 1.0) / 3.0)) for x in f]
        f = [x * s + x / 16.0 * (1.0 - s) for x, s in zip(f, keep)]
    return f


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = dict(c)
    if c["op"] == "rotary":
        t, d = c["tokens"], c["dim"]
        # queries and keys are views of one q, k, v result
        qkv = _rows(gen, t, (c["q_heads"] + 2 * c["heads"]) * d).to(_dtype(c["x"]))
        s["q_in"] = qkv[:, :c["q_heads"] * d].view(t, c["q_heads"], d)
        s["k_in"] = qkv[:, c["q_heads"] * d:(c["q_heads"] + c["heads"]) * d].view(t, c["heads"], d)
        s["positions"] = torch.randint(0, c["far"], (t,), generator=gen, device=DEV, dtype=torch.int32)
        s["f"] = torch.tensor(_frequencies(c), dtype=torch.float64, device=DEV)
        s["gain"] = 0.1 * math.log(16.0) + 1.0 if c["scaling"] == "bands" else 1.0
        if own:
            import tenant_serving_amd as bd
            s["angles"] = bd.bd_rotary_angles(c["turned"], BASE, interleaved=c["interleaved"], scaling=c["scaling"], factor=16.0, trained=TRAINED, gain=s["gain"], device=DEV)
        return s
    if c["op"] == "cache":
        t, row = c["tokens"], c["heads"] * c["dim"]
        pages = -(-t // c["page"]) + 5
        s["kind"] = "e2m1"
        s["cache"] = _cache(s, gen, pages)
        # whole pages in any order, as an allocator hands them out, the tokens in order within them
        order = torch.randperm(pages, generator=gen, device=DEV)
        pos = torch.arange(t, device=DEV)
        s["slots"] = (order[pos // c["page"]] * c["page"] + pos % c["page"]).to(torch.int32)
        # keys and values are views of one q, k, v result with 8 query heads
        qkv = _rows(gen, t, 8 * c["dim"] + 2 * row).to(_dtype(c["x"]))
        s["k_in"] = qkv[:, 8 * c["dim"]:8 * c["dim"] + row].view(t, c["heads"], c["dim"])
        s["v_in"] = qkv[:, 8 * c["dim"] + row:].view(t, c["heads"], c["dim"])
        s["kv"] = _handle(s, s["cache"])
        return s
    new, lens = _lengths(c)
    used = [-(-n // c["page"]) for n in lens]
    s["cache"] = _cache(c, gen, sum(used) + 5)
    order = torch.randperm(sum(used) + 5, generator=gen, device=DEV).to(torch.int32)
    columns = torch.arange(max(used), device=DEV)
    count = torch.tensor(used, device=DEV)
    start = torch.cumsum(count, 0) - count
    at = (start[:, None] + columns[None, :]).clamp(max=sum(used) - 1)
    s["table"] = torch.where(columns[None, :] < count[:, None], order[at], -1).to(torch.int32)  # no page behind the last
    s["lengths"] = torch.tensor(lens, device=DEV, dtype=torch.int32)
    s["q_in"] = (2 * torch.randn((sum(new), c["q_heads"], c["dim"]), generator=gen, device=DEV)).to(_dtype(c.get("q", "bfloat16")))
    ranges = _ranges(c)
    s["first"] = torch.tensor([x for a, _ in ranges for x in a], device=DEV, dtype=torch.int32)
    s["last"] = torch.tensor([x for _, b in ranges for x in b], device=DEV, dtype=torch.int32)
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s["starts"] = torch.tensor(starts, device=DEV, dtype=torch.int32)
    s["new"], s["lens"] = new, lens
    # slopes fall from 1/2 to 1/256 over the heads
    s["slope"] = torch.exp2(-8 * (torch.arange(c["q_heads"], device=DEV, dtype=torch.float64) + 1) / c["q_heads"]).float() if c["slopes"] else None
    s["kv"] = _handle(c, s["cache"])
    return s


# ----------------------------------------------------------------------------
# one pass

def _turn(s, x):
    r = s["turned"]
    angle = s["positions"].double()[:, None, None] * s["f"]
    cos, sin = (torch.cos(angle) * s["gain"]).float(), (torch.sin(angle) * s["gain"]).float()
    x = x.float()
    head, rest = x[..., :r], x[..., r:]
    if s["interleaved"]:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = head[..., :r // 2], head[..., r // 2:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, rest), -1).to(torch.bfloat16)


def _write_read(s):
    page, at = s["slots"].long() // s["page"], s["slots"].long() % s["page"]
    cache, out = s["cache"], {}
    for name in ("k", "v"):
        codes, e = _quantise4(s[name + "_in"].float())
        cache[name][page, :, at] = codes
        cache[name + "_exp"][page, :, :, at] = e
    for name in ("k", "v"):
        out[name] = _held4(cache[name][page, :, at], cache[name + "_exp"][page, :, :, at]).to(torch.bfloat16)
    return out


def _whole(s, name, table):
    """[..., heads, positions, dim] of a cache's array in fp32, by the pages of a table."""
    x = s["cache"][name][table]
    if s["kind"] == "bfloat16":
        x = x.float()
    elif s["kind"] == "e4m3":
        x = s["cache"][name].view(torch.uint8)[table].view(torch.float8_e4m3fn).float() * _power(s["cache"][name + "_exp"][table]).unsqueeze(-1)
    else:
        x = _held4(x, s["cache"][name + "_exp"][table].transpose(-1, -2))
    return x.transpose(-3, -4).flatten(-3, -2)


def _weigh(s, score, v, first, last, position, slope):
    """Outputs from scores [..., keys]: first, last and position broadcast against them."""
    j = torch.arange(score.shape[-1], device=score.device)
    if s["cap"]:
        score = s["cap"] * torch.tanh(score / s["cap"])
    if slope is not None:
        score = score - slope * (position - j).abs()
    score = score.masked_fill(~((j >= first) & (j < last)), -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top.masked_fill(top == -math.inf, 0.0))
    return torch.matmul(p, v) / p.sum(-1, keepdim=True).clamp(min=1e-30)  # a row that sees nothing gives zeros


def _attend(s):
    table = s["table"].long().clamp(min=0)
    b, group = s["batch"], s["q_heads"] // s["heads"]
    k, v = _whole(s, "k", table), _whole(s, "v", table)
    q = s["q_in"].float().view(b, s["heads"], group, s["dim"]) * s["dim"] ** -0.5
    score = torch.matmul(q, k.transpose(2, 3).contiguous())
    slope = None if s["slope"] is None else s["slope"].view(s["heads"], group, 1)
    first, last = (s[x].view(b, 1, 1, 1) for x in ("first", "last"))
    return _weigh(s, score, v, first, last, last - 1, slope).view(b, s["q_heads"], s["dim"]).to(torch.bfloat16)


def _prompt(s):
    group, out = s["q_heads"] // s["heads"], torch.empty_like(s["q_in"])
    begin = 0
    for b, (n, length) in enumerate(zip(s["new"], s["lens"])):
        if n == 0:
            continue
        own_rows = slice(begin, begin + n)
        begin += n
        table = s["table"][b, :-(-length // s["page"])].long()
        k, v = _whole(s, "k", table), _whole(s, "v", table)
        first, last = s["first"][own_rows, None, None], s["last"][own_rows, None, None]
        position = torch.arange(length - n, length, device=DEV)[:, None, None]
        for h in range(s["heads"]):
            heads = slice(h * group, h * group + group)
            q = s["q_in"][own_rows, heads].float() * s["dim"] ** -0.5
            score = torch.matmul(q, k[h].t().contiguous())
            slope = None if s["slope"] is None else s["slope"][heads, None]
            out[own_rows, heads] = _weigh(s, score, v[h], first, last, position, slope).to(torch.bfloat16)
    return out


def run(state):
    s = state
    if own:
        import tenant_serving_amd as bd
        if s["op"] == "rotary":
            return bd.bd_rotary(s["angles"], s["q_in"], s["positions"], s["k_in"])
        if s["op"] == "cache":
            bd.bd_kv_write(s["kv"], s["k_in"], s["v_in"], s["slots"])
            k, v = bd.bd_kv_read(s["kv"], s["slots"])
            return {"k": k, "v": v}
        cap = s["cap"] or None
        if s["op"] == "attend":
            first = s["first"] if s["window"] else None
            return bd.bd_attend(s["q_in"], s["kv"], s["table"], s["lengths"], cap=cap, slopes=s["slope"], first=first)
        first = s["first"] if s["form"] in ("window", "documents") else None
        last = s["last"] if s["form"] == "prefix" else None
        return bd.bd_attend_prompt(s["q_in"], s["kv"], s["table"], s["lengths"], s["starts"], cap=cap, slopes=s["slope"], first=first, last=last)
    if s["op"] == "rotary":
        return _turn(s, s["q_in"]), _turn(s, s["k_in"])
    if s["op"] == "cache":
        return _write_read(s)
    return _attend(s) if s["op"] == "attend" else _prompt(s)


# ----------------------------------------------------------------------------
# the same in 64 bits

def _two_to(e):
    """2^e in float64 for whole e, exactly (a device's pow need not be)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _to_e2m1(x):
    """float64 [..., dim] rounded to what its groups of 32 hold: the nearest of the eight magnitudes times the scale,
    of two that are equally near the one whose code is even."""
    y = x.unflatten(-1, (-1, 32))
    top = y.abs().amax(-1, keepdim=True).clamp(min=6 * 2.0 ** -125)
    e = torch.frexp(top / 6).exponent - 1
    scale = _two_to(torch.where(6 * _two_to(e) < top, e + 1, e))
    m = y.abs() / scale
    held = torch.zeros_like(m)
    for code in range(1, 8):
        mid = (_E2M1[code] + _E2M1[code - 1]) / 2
        held = torch.where((m > mid) | ((m == mid) & (code % 2 == 0)), _E2M1[code], held)
    return (held * scale * torch.sign(y)).flatten(-2)


def _values(s, name, pages):
    """[heads, positions, dim] of some pages in float64."""
    x = torch.index_select(s["cache"][name].view(torch.uint8) if s["kind"] == "e4m3" else s["cache"][name], 0, pages)
    if s["kind"] == "bfloat16":
        x = x.double()
    else:
        e = torch.index_select(s["cache"][name + "_exp"], 0, pages).to(torch.int64) - 127
        if s["kind"] == "e4m3":
            x = x.view(torch.float8_e4m3fn).double() * _two_to(e)[..., None]
        else:
            x = torch.stack((x.bitwise_and(15), x.bitwise_right_shift(4)), -1).flatten(-2).to(torch.int64)
            size = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)[x % 8]
            x = torch.where(x >= 8, -size, size) * _two_to(e).transpose(2, 3).repeat_interleave(32, 3)
    return x.permute(1, 0, 2, 3).flatten(1, 2)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "rotary":
        got = []
        f = torch.tensor(_frequencies(case), dtype=torch.float64, device=DEV)
        for x in (s["q_in"].double(), s["k_in"].double()):
            y, r = x.clone(), s["turned"]
            for i in range(r // 2):
                a, b = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + r // 2)
                t = (s["positions"].double() * f[i])[:, None]
                y[..., a] = s["gain"] * (x[..., a] * torch.cos(t) - x[..., b] * torch.sin(t))
                y[..., b] = s["gain"] * (x[..., b] * torch.cos(t) + x[..., a] * torch.sin(t))
            got.append(y)
        return tuple(got)
    if s["op"] == "cache":
        return {"k": _to_e2m1(s["k_in"].double()), "v": _to_e2m1(s["v_in"].double())}
    group, rows = s["q_heads"] // s["heads"], []
    slope = None if s["slope"] is None else s["slope"].double()
    begin = 0
    for b, (n, length) in enumerate(zip(*_lengths(case))):
        q = s["q_in"][begin:begin + n].double()
        first, last = (s[x][begin:begin + n].to(torch.int64) for x in ("first", "last"))
        begin += n
        if n == 0 or length == 0:
            rows.append(torch.zeros_like(q))
            continue
        pages = s["table"][b, : -(-length // s["page"])]
        k, v = (_values(s, name, pages)[:, :length] for name in ("k", "v"))
        j = torch.arange(length, device=DEV)
        far = (torch.arange(length - n, length, device=DEV)[:, None] - j[None, :]).abs()
        hidden = (j[None, :] < first[:, None]) | (j[None, :] >= last[:, None])
        out = torch.empty_like(q)
        for h in range(s["q_heads"]):
            score = torch.mm(q[:, h].contiguous(), k[h // group].t().contiguous()) / math.sqrt(s["dim"])
            if s["cap"]:
                score = torch.tanh(score / s["cap"]) * s["cap"]
            if slope is not None:
                score -= slope[h] * far
            score[hidden] = -math.inf
            out[:, h] = torch.mm(torch.nan_to_num(torch.softmax(score, 1), nan=0.0), v[h // group])
        rows.append(out)
    return torch.cat(rows)
