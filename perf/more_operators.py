"""The operators of a serving step over a paged KV cache whose models look at a window of
the past: attention with a sliding window and a few first tokens that stay visible, the
blocks of the cache handed out and given back on the GPU, and the rotation of queries and
keys whose positions have several axes. For each one a plain form in elementary torch
operations, the framework's own call, and its definition in 64 bits.

A case names its operator in "op":
  window   attention of the current tokens over the fp16 or the 8-bit cache: a token at
           position p attends position j <= p if j > p - window or j < sinks
  blocks   block tables and slot maps from the lengths of the requests; "back": the blocks
           are given back in a second call, so that every pass starts from the same pool
  rotate   norm of every query and key head and rotary embedding by positions of several axes
  store    the same, keys and values into the 8-bit cache, the rows read back

The 8-bit cache holds, for every token and kv head, e4m3 codes and one biased
power-of-two exponent: e is the least integer >= -32 with max |x| <= 448 * 2^e.
"""
import math
import random

import torch

own = False

_DEV = "cuda" if torch.cuda.is_available() else "cpu"
_E_MIN = -32
_TABLE = 16384  # positions of the rotary table


def listed():
    return [
        # one sequence, one new token: nothing but latency
        dict(name="window one token", op="window", bits=16, batch=1, q_lo=1, q_hi=1, ctx_lo=4096, ctx_hi=4096,
             window=1024, sinks=4, heads=32, kv_heads=8, dim=128, block=128, lens=1),
        # one decode step of 64 sequences, most of them longer than the window
        dict(name="window decode batch", op="window", bits=16, batch=64, q_lo=1, q_hi=1, ctx_lo=1, ctx_hi=8192,
             window=2048, sinks=4, heads=32, kv_heads=8, dim=128, block=128, lens=2),
        # the same over the 8-bit cache, whose first block stays visible
        dict(name="window decode batch, 8 bits", op="window", bits=8, batch=64, q_lo=1, q_hi=1, ctx_lo=1,
             ctx_hi=8192, window=4096, sinks=64, heads=32, kv_heads=8, dim=128, block=64, lens=3),
        # chains of 5 to 16 drafted tokens
        dict(name="window drafts, 8 bits", op="window", bits=8, batch=32, q_lo=5, q_hi=16, ctx_lo=64, ctx_hi=8192,
             window=1024, sinks=0, heads=32, kv_heads=8, dim=128, block=128, lens=4),
        # whole prompts
        dict(name="window prompts", op="window", bits=16, batch=4, q_lo=1024, q_hi=8192, whole=True, ctx_lo=1,
             ctx_hi=1, window=1024, sinks=4, heads=32, kv_heads=8, dim=128, block=128, lens=5),
        # later parts of long prompts, no shared heads
        dict(name="window prompt parts, 8 bits", op="window", bits=8, batch=8, q_lo=512, q_hi=512, ctx_lo=512,
             ctx_hi=8192, window=2048, sinks=4, heads=32, kv_heads=32, dim=128, block=128, lens=6),
        # a decode step of many requests: a sixteenth of them needs a new block
        dict(name="blocks of a decode step", op="blocks", batch=256, q_lo=1, q_hi=1, ctx_lo=1, ctx_hi=4096,
             window=0, sinks=0, block=16, back=False, lens=7),
        # prompts admitted, and their blocks given back when they are done
        dict(name="blocks of prompts, given back", op="blocks", batch=64, q_lo=1, q_hi=4096, whole=True, ctx_lo=1,
             ctx_hi=1, window=0, sinks=0, block=16, back=True, lens=8),
        # one new token of a sequence that holds images
        dict(name="rotate one token, three axes", op="rotate", tokens=1, heads=32, kv_heads=8, dim=128, rot=128,
             sections="16 24 24", cyclic=False, norm=True, interleaved=False, packed=True, lens=9),
        # a video of 16384 patches through one layer
        dict(name="rotate a video", op="rotate", tokens=16384, heads=32, kv_heads=8, dim=128, rot=128,
             sections="24 20 20", cyclic=True, norm=True, interleaved=False, packed=True, lens=10),
        # one decode step of 64 sequences
        dict(name="store a decode step, three axes", op="store", batch=64, q_lo=1, q_hi=1, ctx_lo=1, ctx_hi=4096,
             heads=32, kv_heads=8, dim=128, rot=128, sections="16 24 24", cyclic=False, norm=True,
             interleaved=False, block=128, lens=11),
        # prompts with images among their text
        dict(name="store prompts with images", op="store", batch=8, q_lo=1, q_hi=2048, ctx_lo=1, ctx_hi=4096,
             heads=32, kv_heads=8, dim=128, rot=128, sections="16 24 24", cyclic=False, norm=True,
             interleaved=False, block=64, lens=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "window", "window", "blocks", "rotate", "store"])
    heads, kv_heads = rng.choice([(32, 8), (32, 32), (40, 40), (16, 1), (28, 4), (8, 2), (6, 3)])
    dim = rng.choice([64, 128, 128, 256])
    block = rng.choice([16, 32, 48, 64, 128])
    lens = rng.randrange(1 << 30)
    if op in ("rotate", "store"):
        rot = rng.choice([dim, dim, dim // 2])
        pairs, axes = rot // 2, rng.choice([2, 3, 3, 3, 4])
        cyclic = rng.random() < 0.5
        if cyclic:  # every axis but the first in every axes-th place, as far as it goes
            part = [rng.randint(0, pairs // axes) for _ in range(axes - 1)]
        else:
            cut = sorted(rng.randint(0, pairs) for _ in range(axes - 1))
            part = [b - a for a, b in zip(cut, cut[1:] + [pairs])]
        rotary = dict(rot=rot, sections=" ".join(map(str, [pairs - sum(part)] + part)), cyclic=cyclic,
                      norm=rng.random() < 0.75, interleaved=rng.random() < 0.4, lens=lens)
    if op == "rotate":
        room = 16384 * 40 * 128 // ((heads + kv_heads) * dim)
        return dict(op=op, tokens=_log_int(rng, 1, room), heads=heads, kv_heads=kv_heads, dim=dim,
                    packed=rng.random() < 0.7, **rotary)
    batch = _log_int(rng, 1, 64)
    if op == "store":
        q_hi = _log_int(rng, 1, max(1, 8192 * 48 * 128 // ((2 * kv_heads + heads) * dim * batch)))
        return dict(op=op, batch=batch, q_lo=rng.choice([1, q_hi]), q_hi=q_hi, ctx_lo=1,
                    ctx_hi=max(q_hi, _log_int(rng, 16, 4096)), heads=heads, kv_heads=kv_heads, dim=dim,
                    block=block, **rotary)
    window = _log_int(rng, 1, 8192)
    sinks = rng.choice([0, 1, 4, 64, _log_int(rng, 1, 1024)])
    if op == "blocks":
        batch, back = _log_int(rng, 1, 512), rng.random() < 0.5
        if rng.random() < 0.4:
            window = sinks = 0
        q_hi = _log_int(rng, 1, max(1, 131072 // batch))
        return dict(op=op, batch=batch, q_lo=rng.choice([0, 1, q_hi]), q_hi=q_hi, whole=back, ctx_lo=1,
                    ctx_hi=max(q_hi, _log_int(rng, 16, 16384)), window=window, sinks=sinks, block=block, back=back,
                    lens=lens)
    bits = rng.choice([8, 16])
    seen = min(window + sinks, 16384)
    rows = max(1, 10 ** 11 // (4 * heads * dim * seen))  # of all sequences
    if rng.random() < 0.6:  # decode steps and drafts
        q_hi = min(_log_int(rng, 1, 64), max(1, rows // batch))
    else:  # prompts
        batch = min(batch, 16)
        q_hi = _log_int(rng, 16, max(16, min(4096, rows // batch)))
    room = 64 * 1024 * 8 * 128 // (kv_heads * dim)
    return dict(op=op, bits=bits, batch=batch, q_lo=rng.choice([1, q_hi]), q_hi=q_hi, whole=rng.random() < 0.2,
                ctx_lo=1, ctx_hi=max(q_hi, _log_int(rng, 16, max(16, min(32768, room // batch)))), window=window,
                sinks=sinks, heads=heads, kv_heads=kv_heads, dim=dim, block=block, lens=lens)


def _lengths(case):
    """(query lengths, context lengths) of the case's sequences."""
    rng = random.Random(case["lens"])
    q = [rng.randint(case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    ctx = [max(n, rng.randint(case["ctx_lo"], case["ctx_hi"])) for n in q]
    return (q, list(q)) if case.get("whole") else (q, ctx)


def _sections(case):
    """How many pairs turn by the position of each axis."""
    return tuple(int(n) for n in case["sections"].split())


def _first_page(case, q, ctx):
    """The first block behind the sinks of which a current or later token sees anything."""
    return max(0, ctx - q - case["window"] + 1) // case["block"] if case["window"] else 0


# ---- inputs

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=_DEV, dtype=torch.float32)


def _keys(gen, *shape):
    """Keys as models make them: a few dims of a head are much larger than the rest."""
    gain = 1 + 4 * (torch.rand(shape[-2:], generator=gen, device=_DEV) > 0.97)
    return (_normal(gen, *shape) * gain).half()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=_DEV)


def _tables(gen, ctx, block, first=None, kept=0):
    """Block tables and the blocks there are; of a sequence whose `first` block is given, those
    between its `kept` first ones and that one have gone back and read -1."""
    need = _ints([-(-n // block) for n in ctx])[:, None]
    cols = int(need.max()) + 1
    i = torch.arange(cols, device=_DEV)
    live = i < need
    if first is not None:
        live &= (i < kept) | (i >= _ints(first)[:, None])
    used = int(live.sum())
    total = used + max(1, used // 10)
    order = torch.randperm(total, generator=gen, device=_DEV).to(torch.int32)
    tables = torch.full(live.shape, -1, dtype=torch.int32, device=_DEV)
    tables[live] = order[:used]
    return tables, total, order[used:]


def _positions(case, q, starts):
    """Positions [axes, tokens] of text and images in turn: a text token's are the same on every
    axis, an image's patches have the time of its place and a place of their own on the others."""
    rng = random.Random(case["lens"] + 1)
    axes = len(_sections(case))
    rows = [[] for _ in range(axes)]
    for n, start in zip(q, starts):
        at = start
        while n > 0:
            if rng.random() < 0.5 or n < 16:
                k = min(n, rng.randint(1, 256))
                for row in rows:
                    row.extend(range(at, at + k))
                at += k
            else:
                h, w = rng.randint(2, 32), rng.randint(2, 32)
                k = min(n, h * w * rng.randint(1, 4))
                for a, row in enumerate(rows):
                    row.extend(at + (i // (h * w) if a == 0 else i // w % h if a == 1 else i % w)
                               for i in range(k))
                at += max(h, w)
            n -= k
    return torch.tensor(rows, dtype=torch.int32, device=_DEV) % _TABLE


def _rotary(gen, s, case):
    dim, rot = case["dim"], case["rot"]
    s["q_weight"] = (1 + 0.1 * _normal(gen, dim)).half() if case["norm"] else None
    s["k_weight"] = (1 + 0.1 * _normal(gen, dim)).half() if case["norm"] else None
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device=_DEV, dtype=torch.float64) / rot)
    angle = torch.arange(_TABLE, device=_DEV, dtype=torch.float64)[:, None] * freq
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()


def _heads(gen, tokens, h, hk, dim, packed, values):
    """Query, key (and value) of a packed projection, or tensors of their own."""
    x = _normal(gen, tokens, h + 2 * hk, dim).half()
    parts = [x[:, :h], x[:, h:h + hk], x[:, h + hk:]][:3 if values else 2]
    return [p if packed else p.contiguous() for p in parts]


def prepare(case, seed):
    gen = torch.Generator(device=_DEV).manual_seed(int(seed))
    s = dict(case=case)
    if own:
        import paged_kv_cache_206_gb300 as pa
    if case["op"] == "rotate":
        t = case["tokens"]
        _rotary(gen, s, case)
        s["q"], s["k"] = _heads(gen, t, case["heads"], case["kv_heads"], case["dim"], case["packed"], False)
        s["positions"] = _positions(case, [t], [int(seed) % 4096])
        s["q_out"] = torch.empty((t, case["heads"], case["dim"]), dtype=torch.float16, device=_DEV)
        s["k_out"] = torch.empty((t, case["kv_heads"], case["dim"]), dtype=torch.float16, device=_DEV)
        return s
    q, ctx = _lengths(case)
    bs = case["block"]
    s["ctx"], s["qlen"] = _ints(ctx), _ints(q)
    s["q_start"] = _ints([sum(q[:b]) for b in range(len(q))])
    total, s["max_q"], s["max_ctx"] = sum(q), max(q), max(ctx)
    if case["op"] == "blocks":
        # as the step before left the pool: without the current tokens, and without what has
        # left the window since
        old = [c - n for n, c in zip(q, ctx)]
        cols = -(-s["max_ctx"] // bs) + 1
        kept = -(-case["sinks"] // bs)
        held = [-(-n // bs) for n in old]
        first = [min(_first_page(case, 1, n), h) if n else 0 for n, h in zip(old, held)]
        gone = [max(0, f - kept) for f in first]
        free = sum(-(-n // bs) - h for n, h in zip(ctx, held))
        live = sum(h - g for h, g in zip(held, gone))
        blocks = live + free + max(1, (live + free) // 10)
        order = torch.randperm(blocks, generator=gen, device=_DEV).to(torch.int32)
        i = torch.arange(cols, device=_DEV)
        there = (i < _ints(held)[:, None]) & ((i < kept) | (i >= kept + _ints(gone)[:, None]))
        s["tables"] = torch.full((len(q), cols), -1, dtype=torch.int32, device=_DEV)
        s["tables"][there] = order[:live]
        s["free"] = torch.cat([order[live:], torch.zeros(live, dtype=torch.int32, device=_DEV)])
        s["count"] = _ints([blocks - live])
        s["held"], s["gone"] = _ints(held), _ints(gone)
        s["slots"] = torch.empty(total, dtype=torch.int64, device=_DEV)
        s["positions"] = torch.empty(total, dtype=torch.int32, device=_DEV)
        s["none"] = torch.zeros_like(s["ctx"])
        if own:
            s["pool"] = pa.BlockPool(s["tables"], s["held"], s["gone"], s["free"], s["count"], block_size=bs,
                                     window=case["window"], sinks=case["sinks"])
        return s
    hk, dim = case["kv_heads"], case["dim"]
    if case["op"] == "window":
        first = [_first_page(case, n, c) for n, c in zip(q, ctx)]
        s["tables"], blocks, _ = _tables(gen, ctx, bs, first, -(-case["sinks"] // bs))
        s["key"], s["value"] = _keys(gen, blocks, bs, hk, dim), _normal(gen, blocks, bs, hk, dim).half()
        s["key_exps"] = s["value_exps"] = None
        if case["bits"] == 8:
            s["key"], s["key_exps"] = _quantise_blocks(s["key"])
            s["value"], s["value_exps"] = _quantise_blocks(s["value"])
        s["q"] = _normal(gen, total, case["heads"], dim).half()
        s["out"] = torch.empty_like(s["q"])
        if own:
            s["step"] = pa.WindowStep(s["key"], s["value"], s["key_exps"], s["value_exps"], batch=len(q),
                                      num_heads=case["heads"], max_seqlen_q=s["max_q"],
                                      max_blocks_per_seq=s["tables"].shape[1], window=case["window"],
                                      sinks=case["sinks"])
        return s
    s["tables"], blocks, _ = _tables(gen, ctx, bs)
    for name in ("key", "value"):
        s[name] = torch.zeros((blocks, bs, hk, dim), dtype=torch.float8_e4m3fn, device=_DEV)
        s[name + "_exps"] = torch.zeros((blocks, hk, bs), dtype=torch.uint8, device=_DEV)
    s["starts"] = s["ctx"] - s["qlen"]
    s["k_out"] = torch.empty((total, hk, dim), dtype=torch.float16, device=_DEV)
    s["v_out"] = torch.empty((total, hk, dim), dtype=torch.float16, device=_DEV)
    _rotary(gen, s, case)
    s["q"], s["k"], s["v"] = _heads(gen, total, case["heads"], hk, dim, True, True)
    s["positions"] = _positions(case, q, [c - n for n, c in zip(q, ctx)])
    s["q_out"] = torch.empty((total, case["heads"], dim), dtype=torch.float16, device=_DEV)
    if own:
        s["cache"] = pa.QuantCache(s["key"], s["value"], s["key_exps"], s["value_exps"])
    return s


# ---- plain forms

def _quantise(x):
    """(e4m3 codes, exponents) of fp32 rows."""
    top = torch.where(x.isfinite(), x.abs(), torch.zeros_like(x)).amax(-1)
    m, k = torch.frexp(top)
    e = torch.where(m <= 0.875, k - 9, k - 8).clamp(min=_E_MIN)
    e = torch.where(top > 0, e, torch.full_like(e, _E_MIN))
    y = torch.ldexp(x, -e[..., None])
    return y.to(torch.float8_e4m3fn), e


def _quantise_blocks(x):
    """The cache [blocks, bs, Hk, D] in 8 bits, with its exponents [blocks, Hk, bs]."""
    step = max(1, (1 << 26) // x[0].numel())
    parts = [_quantise(p.float()) for p in x.split(step)]
    return (torch.cat([c for c, _ in parts]),
            torch.cat([(e + 127).to(torch.uint8).transpose(1, 2) for _, e in parts]).contiguous())


def _held(cache, exps, block, place):
    """The fp32 values that the cache holds at these places."""
    if exps is None:
        return cache[block, place].float()
    x = cache.view(torch.uint8)[block, place].view(torch.float8_e4m3fn).float()
    return torch.ldexp(x, exps.transpose(1, 2)[block, place].int()[..., None] - 127)


def _window(s):
    """Pieces of up to 128 tokens of a sequence, as many at a time as a gigabyte of scores holds:
    the sinks and the keys from the first one's window on are gathered and attended."""
    case, q = s["case"], s["q"]
    window, sinks, bs = case["window"], case["sinks"], case["block"]
    hk, group, dim = case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"]
    piece = min(s["max_q"], 128)
    n_q, n_ctx = _lengths(case)
    pieces = [(b, i) for b, n in enumerate(n_q) for i in range(0, n, piece)]
    near = min(window + piece - 1, s["max_ctx"])
    far = min(sinks, s["max_ctx"])
    step = max(1, (1 << 28) // (piece * case["heads"] * (near + far) + (near + far) * hk * dim))
    out = s["out"]
    for at in range(0, len(pieces), step):
        b, i0 = torch.tensor(pieces[at:at + step], device=q.device).unbind(1)
        ctx, qlen = s["ctx"].long()[b], s["qlen"].long()[b]
        i = i0[:, None] + torch.arange(piece, device=q.device)
        live = i < qlen[:, None]
        rows = (s["q_start"].long()[b][:, None] + i)[live]
        pos = (ctx - qlen)[:, None] + i
        # the sinks, then `near` keys from the first row's window on (sinks among them only once)
        lo = (pos[:, :1] - window + 1).clamp(min=0)
        key = torch.cat([torch.arange(far, device=q.device).expand(len(b), far),
                         lo + torch.arange(near, device=q.device)], 1)
        there = key < ctx[:, None]
        there[:, far:] &= key[:, far:] >= far
        page = torch.where(there, key, torch.zeros_like(key)) // bs
        block = torch.gather(s["tables"].long()[b], 1, page).clamp(min=0)
        k = _held(s["key"], s["key_exps"], block, key % bs)
        v = _held(s["value"], s["value_exps"], block, key % bs)
        seen = there[:, None] & (key[:, None] <= pos[..., None]) & (
            (key[:, None] > pos[..., None] - window) | (key[:, None] < sinks))
        seen = (seen & live[..., None])[:, None, :, None]
        x = torch.zeros((len(b), piece) + q.shape[1:], device=q.device)
        x[live] = q[rows].float()
        x = x.view(len(b), piece, hk, group, dim).permute(0, 2, 1, 3, 4).flatten(2, 3)
        score = torch.matmul(x, k.permute(0, 2, 3, 1)) / math.sqrt(dim)
        score = score.unflatten(2, (piece, group)).masked_fill(~seen, -math.inf).flatten(2, 3)
        p = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-1e30))
        p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
        o = torch.matmul(p, v.permute(0, 2, 1, 3))
        o = o.view(len(b), hk, piece, group, dim).permute(0, 2, 1, 3, 4).flatten(2, 3)
        out[rows] = o[live].half()
    return out


def _blocks(s, ctx, qlen):
    """One step of the pool: blocks given back, then blocks handed out, then the tokens' slots."""
    case, tables, free, count = s["case"], s["tables"], s["free"], s["count"]
    bs, kept = case["block"], -(-case["sinks"] // case["block"])
    i = torch.arange(tables.shape[1], device=tables.device)
    held, gone = s["held"].long()[:, None], s["gone"].long()[:, None]
    live = (i < held) & ((i < kept) | (i >= kept + gone))
    lens, q = ctx.long()[:, None], qlen.long()[:, None]
    if case["window"]:
        first = torch.minimum((lens - q - case["window"] + 1).clamp(min=0) // bs, held)
    else:
        first = torch.zeros_like(held)
    back = live & ((lens == 0) | ((i >= kept) & (i < first)))
    some = lens > 0
    need = (lens + bs - 1) // bs
    more = (i >= held) & (i < need)
    n = count.long()
    # given back: the first one comes to lie on top; handed out: the top first
    nth = (back.flatten().long().cumsum(0) - 1).view(back.shape)
    n_back = back.sum()
    free[(n + n_back - 1 - nth)[back]] = tables[back]
    tables[back] = -1
    nth = (more.flatten().long().cumsum(0) - 1).view(more.shape)
    top = n + n_back
    got = more & (nth < top)
    tables[got] = free[(top - 1 - nth)[got]]
    count.copy_((top - got.sum()).to(torch.int32))
    s["held"].copy_(torch.where(some, held + got.sum(1, keepdim=True), torch.zeros_like(held))[:, 0])
    s["gone"].copy_(torch.where(some, torch.maximum(gone, first - kept), torch.zeros_like(gone))[:, 0])
    slots, positions = s["slots"], s["positions"]
    slots.fill_(-1)
    positions.fill_(-1)
    t = torch.arange(slots.shape[0], device=tables.device)
    end = qlen.long().cumsum(0)
    b = torch.searchsorted(end, t, right=True)
    mine = b < len(end)
    t, b = t[mine], b[mine]
    pos = ctx.long()[b] - end[b] + t
    block = tables.long()[b, pos // bs]
    positions[t] = pos.to(torch.int32)
    slots[t] = torch.where(block >= 0, block * bs + pos % bs, torch.full_like(pos, -1))


def _axis_of(case):
    """The axis whose position turns pair i, for every pair."""
    sections, axes, pairs = _sections(case), len(_sections(case)), case["rot"] // 2
    if not case["cyclic"]:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    return [i % axes if i < axes * sections[i % axes] else 0 for i in range(pairs)]


def _rotate(s, x, weight):
    case = s["case"]
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * weight.float()
    rot = case["rot"]
    axis = torch.tensor(_axis_of(case), device=x.device)
    pos = s["positions"].long()[axis].t()  # [tokens, pairs]
    pair = torch.arange(rot // 2, device=x.device)
    c, z = s["cos_sin"][pos, pair][:, None], s["cos_sin"][pos, rot // 2 + pair][:, None]
    if case["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * c - b * z, b * c + a * z], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * c - b * z, b * c + a * z], -1)
    return torch.cat([turned, y[..., rot:]], -1)


def _current(s):
    """Block and place of every current token."""
    i = torch.arange(s["max_q"], device=s["ctx"].device)
    there = i < s["qlen"][:, None]
    pos = torch.where(there, s["starts"][:, None] + i, torch.zeros_like(i)).long()
    bs = s["case"]["block"]
    return torch.gather(s["tables"].long(), 1, pos // bs)[there], (pos % bs)[there]


def _put(s, name, x):
    block, place = _current(s)
    codes, e = _quantise(x)
    s[name].view(torch.uint8)[block, place] = codes.view(torch.uint8)
    s[name + "_exps"].transpose(1, 2)[block, place] = (e + 127).to(torch.uint8)


def _get(s, name):
    return _held(s[name], s[name + "_exps"], *_current(s)).half()


def run(s):
    op, case = s["case"]["op"], s["case"]
    if op == "blocks":
        if own:
            s["pool"].step(s["ctx"], s["qlen"], s["slots"], s["positions"])
            if case["back"]:
                s["pool"].step(s["none"], s["none"])
        else:
            _blocks(s, s["ctx"], s["qlen"])
            if case["back"]:
                slots, positions = s["slots"].clone(), s["positions"].clone()
                _blocks(s, s["none"], s["none"])
                s["slots"], s["positions"] = slots, positions
        return tuple(s[name] for name in ("tables", "held", "gone", "free", "count", "slots", "positions"))
    if own:
        import paged_kv_cache_206_gb300 as pa
        if op == "window":
            return s["step"].run(s["q"], s["tables"], s["ctx"], s["qlen"], s["out"])
        if op == "rotate":
            pa.pa_qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["cos_sin"], s["positions"],
                               s["q_out"], s["k_out"], eps=1e-6, interleaved=case["interleaved"],
                               sections=_sections(case), cyclic=case["cyclic"])
            return s["q_out"], s["k_out"]
        s["cache"].store(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["cos_sin"], s["positions"],
                         s["tables"], s["ctx"], s["qlen"], s["max_q"], s["q_out"], eps=1e-6,
                         interleaved=case["interleaved"], sections=_sections(case), cyclic=case["cyclic"])
        s["cache"].read(s["tables"], s["starts"], s["ctx"], s["q_start"], s["max_q"], s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"], s["q_out"]
    if op == "window":
        return _window(s)
    if op == "rotate":
        return _rotate(s, s["q"], s["q_weight"]).half(), _rotate(s, s["k"], s["k_weight"]).half()
    turned = _rotate(s, s["q"], s["q_weight"]).half()
    _put(s, "key", _rotate(s, s["k"], s["k_weight"]))
    _put(s, "value", s["v"].float())
    return _get(s, "key"), _get(s, "value"), turned


def _pairs(case, q, ctx):
    """(keys that a sequence's tokens see between them, pairs of token and key)."""
    window, sinks = case["window"], case["sinks"]
    lo = max(0, ctx - q - window + 1)
    keys = ctx - lo + min(sinks, lo) if q else 0
    pairs = 0
    for p in range(ctx - q, ctx):
        first = max(0, p - window + 1)
        pairs += p + 1 - first + min(sinks, first)
    return keys, pairs


def work(case):
    if case["op"] == "rotate":
        n = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        return dict(bytes=n * 4 + case["tokens"] * (case["rot"] * 4 + 4 * len(_sections(case))), flops=n * 8)
    q, ctx = _lengths(case)
    if case["op"] == "blocks":
        # lengths and the state in and out, a block taken (and given back) and its entry, slots and positions
        bs = case["block"]
        new = sum(-(-c // bs) - -(-(c - n) // bs) for n, c in zip(q, ctx))
        b = len(q) * 24 + new * 8 + sum(q) * 12
        return dict(bytes=b + (len(q) * 24 + new * 8 if case["back"] else 0), flops=4 * sum(q) + 16 * len(q))
    hk, dim = case["kv_heads"], case["dim"]
    if case["op"] == "window":
        seen = [_pairs(case, n, c) for n, c in zip(q, ctx)]
        row = dim * 2 if case["bits"] == 16 else dim + 1
        return dict(bytes=sum(k for k, _ in seen) * hk * 2 * row + sum(q) * case["heads"] * dim * 4,
                    flops=4 * case["heads"] * dim * sum(p for _, p in seen))
    n = sum(q) * hk * 2  # read, written in 8 bits, and given back in 16
    m = sum(q) * case["heads"] * dim
    return dict(bytes=n * (dim * 5 + 1) + m * 4 + sum(q) * (case["rot"] * 4 + 4 * len(_sections(case))),
                flops=n * dim * 8 + m * 8)


# ---- the definitions in 64 bits

def _exact_rows(s, x, weight):
    case, rot = s["case"], s["case"]["rot"]
    y = x.double()
    if weight is not None:
        y = y / ((y ** 2).sum(-1, keepdim=True) / y.shape[-1] + 1e-6).sqrt() * weight.double()
    out = y.clone()
    left = list(_sections(case))
    for i in range(rot // 2):
        if case["cyclic"]:
            axis = i % len(left)
            axis = axis if axis and i // len(left) < _sections(case)[axis] else 0
        else:
            axis = next(a for a, n in enumerate(left) if n)
            left[axis] -= 1
        lo, hi = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
        row = s["cos_sin"].double()[s["positions"][axis].long()]
        c, z = row[:, i, None], row[:, rot // 2 + i, None]
        out[..., lo] = y[..., lo] * c - y[..., hi] * z
        out[..., hi] = y[..., lo] * z + y[..., hi] * c
    return out


def _exact_8bit(x):
    """What the 8-bit cache holds for these rows."""
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.ceil(torch.log2(top.clamp(min=1e-300) / 448)).clamp(min=_E_MIN))
    scale = torch.where(scale * 224 >= top, scale / 2, scale).clamp(min=2.0 ** _E_MIN)
    y = x / scale
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step * scale


def _exact_values(s, name, b, keys):
    """Keys or values of these positions of sequence b, [n, Hk, D]."""
    bs = s["case"]["block"]
    block, place = s["tables"][b].long()[keys // bs], keys % bs
    if s[name + "_exps"] is None:
        return s[name][block, place].double()
    codes = s[name].view(torch.uint8)[block, place].view(torch.float8_e4m3fn).double()
    return codes * torch.exp2(s[name + "_exps"][block, :, place].double() - 127)[..., None]


def _exact_window(s):
    case, outs, at = s["case"], [], 0
    group, scale = case["heads"] // case["kv_heads"], case["dim"] ** -0.5
    for b, (n, length) in enumerate(zip(*_lengths(case))):
        for i in range(0, n, 256):
            m = min(256, n - i)
            pos = torch.arange(length - n + i, length - n + i + m, device=s["q"].device)
            keys = torch.arange(int(pos[-1]) + 1, device=s["q"].device)
            keys = keys[(keys > int(pos[0]) - case["window"]) | (keys < case["sinks"])]
            k, v = _exact_values(s, "key", b, keys), _exact_values(s, "value", b, keys)
            rows = s["q"][at + i:at + i + m].double().view(m, case["kv_heads"], group, -1)
            gap = pos[:, None] - keys
            hidden = (gap < 0) | ((gap >= case["window"]) & (keys >= case["sinks"]))
            score = torch.einsum("nhgd,lhd->hgnl", rows, k) * scale
            weight = torch.softmax(score.masked_fill(hidden, -math.inf), -1)
            outs.append(torch.einsum("hgnl,lhd->nhgd", weight, v).reshape(m, case["heads"], -1))
        at += n
    return torch.cat(outs)


def _exact_blocks(s):
    """The pool's step told in lists."""
    case, bs = s["case"], s["case"]["block"]
    tables, held, gone = (s[n].tolist() for n in ("tables", "held", "gone"))
    free, n = s["free"].tolist(), int(s["count"])
    kept = -(-case["sinks"] // bs)
    q, ctx = _lengths(case)
    slots, positions = [], []
    for step in range(2 if case["back"] else 1):
        if step:
            q, ctx = [0] * len(q), [0] * len(ctx)
        back = []
        for b, length in enumerate(ctx):
            if length == 0:
                pages = [i for i in range(held[b]) if i < kept or i >= kept + gone[b]]
                held[b] = gone[b] = 0
            else:
                first = min(_first_page(case, q[b], length), held[b])
                pages = list(range(kept + gone[b], first))
                gone[b] += len(pages)
            back += [tables[b][i] for i in pages]
            for i in pages:
                tables[b][i] = -1
        for block in reversed(back):
            free[n] = block
            n += 1
        for b, length in enumerate(ctx):
            while held[b] * bs < length and n:
                n -= 1
                tables[b][held[b]] = free[n]
                held[b] += 1
            for p in range(length - q[b], length):
                positions.append(p)
                slots.append(tables[b][p // bs] * bs + p % bs if p // bs < held[b] else -1)
    make = lambda v, t=torch.int32: torch.tensor(v, dtype=t, device=s["ctx"].device)  # noqa: E731
    return (make(tables), make(held), make(gone), make(free), make([n]), make(slots, torch.int64),
            make(positions))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "window":
        return None if work(case)["flops"] > 1e12 else _exact_window(s)
    if case["op"] == "blocks":
        return _exact_blocks(s)
    if case["op"] == "rotate":
        return _exact_rows(s, s["q"], s["q_weight"]), _exact_rows(s, s["k"], s["k_weight"])
    return (_exact_8bit(_exact_rows(s, s["k"], s["k_weight"])), _exact_8bit(s["v"]),
            _exact_rows(s, s["q"], s["q_weight"]))
