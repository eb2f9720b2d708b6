"""The operators that surround a paged KV cache in a speculative serving step:
norms and rotation of queries and keys, an 8-bit cache written and read back, and
attention for a tree of drafted tokens over a cache. For each one a plain form in
elementary torch operations, the framework's own call, and its definition in 64 bits.

A case names its operator in "op":
  rotate   norm of every query and key head and rotary embedding, fp16 to fp16
  write    keys and values quantised into the paged cache, and the rows written read back
  store    rotate and write in one pass over a packed QKV projection, rows read back
  read     whole contexts of the 8-bit cache read back to fp16
  tree     attention of drafted tokens over the fp16 or the 8-bit cache

The 8-bit cache holds, for every token and kv head, e4m3 codes and one biased
power-of-two exponent: e is the least integer >= -32 with max |x| <= 448 * 2^e.
"""
import math
import random

import torch

own = False

_DEV = "cuda" if torch.cuda.is_available() else "cpu"
_E_MIN = -32


def listed():
    return [
        # the smallest call of a decode loop: one token's heads, nothing but latency
        dict(name="rotate one token", op="rotate", tokens=1, heads=32, kv_heads=8, dim=128, rot=128,
             norm=True, interleaved=False, packed=True),
        # a prompt of 8192 tokens through one layer
        dict(name="rotate a prompt", op="rotate", tokens=8192, heads=32, kv_heads=8, dim=128, rot=128,
             norm=True, interleaved=False, packed=True),
        # four drafted tokens for each of 32 sequences, no shared heads
        dict(name="write drafts", op="write", batch=32, q_lo=4, q_hi=4, ctx_lo=64, ctx_hi=8192, kv_heads=32,
             dim=128, block=128, lens=1),
        # four prompts of 2048 tokens, no shared heads
        dict(name="write prompts", op="write", batch=4, q_lo=2048, q_hi=2048, ctx_lo=2048, ctx_hi=2048,
             kv_heads=32, dim=128, block=128, lens=2),
        # one decode step of 64 sequences
        dict(name="store a decode step", op="store", batch=64, q_lo=1, q_hi=1, ctx_lo=1, ctx_hi=4096,
             heads=32, kv_heads=8, dim=128, rot=128, norm=True, interleaved=False, block=128, lens=3),
        # prompts of ragged lengths, the later parts of longer contexts among them
        dict(name="store ragged prompts", op="store", batch=8, q_lo=1, q_hi=2048, ctx_lo=1, ctx_hi=4096,
             heads=32, kv_heads=8, dim=128, rot=128, norm=True, interleaved=False, block=64, lens=4),
        # one short context: a single sequence handed over
        dict(name="read a short context", op="read", batch=1, ctx_lo=37, ctx_hi=37, kv_heads=8, dim=128,
             block=16, lens=5),
        # the contexts of a whole batch handed over
        dict(name="read a batch", op="read", batch=32, ctx_lo=64, ctx_hi=8192, kv_heads=8, dim=128,
             block=128, lens=6),
        # one sequence, one new token
        dict(name="tree one token, 8 bits", op="tree", bits=8, batch=1, q_lo=1, q_hi=1, chain=True,
             ctx_lo=4096, ctx_hi=4096, heads=32, kv_heads=8, dim=128, block=128, lens=7),
        # a decode batch without drafts over the 8-bit cache
        dict(name="tree decode batch, 8 bits", op="tree", bits=8, batch=64, q_lo=1, q_hi=1, chain=True,
             ctx_lo=1, ctx_hi=4096, heads=32, kv_heads=8, dim=128, block=128, lens=8),
        # trees of up to 16 drafted tokens over the 8-bit cache
        dict(name="tree of 16, 8 bits", op="tree", bits=8, batch=32, q_lo=5, q_hi=16, chain=False,
             ctx_lo=64, ctx_hi=8192, heads=32, kv_heads=8, dim=128, block=128, lens=9),
        # trees of 64 drafted tokens over the fp16 cache
        dict(name="tree of 64, fp16", op="tree", bits=16, batch=16, q_lo=64, q_hi=64, chain=False,
             ctx_lo=64, ctx_hi=8192, heads=32, kv_heads=8, dim=128, block=128, lens=10),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotate", "write", "store", "read", "tree", "tree", "tree"])
    heads, kv_heads = rng.choice([(32, 8), (32, 32), (40, 40), (16, 1), (28, 4), (8, 2), (6, 3)])
    dim = rng.choice([64, 128, 128, 256])
    block = rng.choice([16, 32, 48, 64, 128])
    lens = rng.randrange(1 << 30)
    rotary = dict(rot=rng.choice([dim, dim, dim // 2]), norm=rng.random() < 0.75,
                  interleaved=rng.random() < 0.4)
    if op == "rotate":
        room = 8192 * 40 * 128 // ((heads + kv_heads) * dim)
        return dict(op=op, tokens=_log_int(rng, 1, room), heads=heads, kv_heads=kv_heads, dim=dim,
                    packed=rng.random() < 0.7, **rotary)
    if op in ("write", "store"):
        batch = _log_int(rng, 1, 64)
        row = (2 * kv_heads + (heads if op == "store" else 0)) * dim
        q_hi = _log_int(rng, 1, max(1, 8192 * 48 * 128 // (row * batch)))
        c = dict(op=op, batch=batch, q_lo=rng.choice([1, q_hi]), q_hi=q_hi, ctx_lo=1,
                 ctx_hi=max(q_hi, _log_int(rng, 16, 4096)), kv_heads=kv_heads, dim=dim, block=block, lens=lens)
        return c if op == "write" else dict(c, heads=heads, **rotary)
    if op == "read":
        room = 128 * 1024 * 8 * 128 // (kv_heads * dim)
        batch = _log_int(rng, 1, 64)
        ctx_hi = _log_int(rng, 1, max(1, min(16384, room // batch)))
        return dict(op=op, batch=batch, ctx_lo=rng.choice([1, ctx_hi]), ctx_hi=ctx_hi, kv_heads=kv_heads,
                    dim=dim, block=block, lens=lens)
    bits = rng.choice([8, 8, 16])
    q_hi = _log_int(rng, 1, 64)
    room = 64 * 1024 * 8 * 128 // (kv_heads * dim)
    batch = _log_int(rng, 1, 64)
    ctx_hi = max(q_hi, _log_int(rng, 16, max(16, min(16384, room // batch))))
    return dict(op=op, bits=bits, batch=batch, q_lo=rng.choice([1, q_hi]), q_hi=q_hi, chain=rng.random() < 0.3,
                ctx_lo=rng.choice([1, ctx_hi]), ctx_hi=ctx_hi, heads=heads, kv_heads=kv_heads, dim=dim,
                block=block, lens=lens)


def _lengths(case):
    """(query lengths, context lengths) of the case's sequences."""
    rng = random.Random(case["lens"])
    q = [rng.randint(case.get("q_lo", 0), case.get("q_hi", 0)) for _ in range(case["batch"])]
    ctx = [max(n, rng.randint(case["ctx_lo"], case["ctx_hi"])) for n in q]
    return q, ctx


# ---- inputs

def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=_DEV, dtype=torch.float32)


def _keys(gen, *shape):
    """Keys as models make them: a few dims of a head are much larger than the rest."""
    gain = 1 + 4 * (torch.rand(shape[-2:], generator=gen, device=_DEV) > 0.97)
    return (_normal(gen, *shape) * gain).half()


def _tables(gen, ctx, block):
    need = [-(-n // block) for n in ctx]
    cols = max(need) + 1
    total = sum(need) + max(1, sum(need) // 10)
    order = torch.randperm(total, generator=gen, device=_DEV)
    at = torch.tensor([sum(need[:b]) for b in range(len(need))], device=_DEV)
    cell = at[:, None] + torch.arange(cols, device=_DEV)
    return order[cell.clamp(max=total - 1)].to(torch.int32), total


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device=_DEV)


def _rotary(gen, s, case):
    dim, rot = case["dim"], case["rot"]
    s["q_weight"] = (1 + 0.1 * _normal(gen, dim)).half() if case["norm"] else None
    s["k_weight"] = (1 + 0.1 * _normal(gen, dim)).half() if case["norm"] else None
    freq = 10000.0 ** (-torch.arange(0, rot, 2, device=_DEV, dtype=torch.float64) / rot)
    angle = torch.arange(16384, device=_DEV, dtype=torch.float64)[:, None] * freq
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()


def _heads(gen, tokens, h, hk, dim, packed, values):
    """Query, key (and value) of a packed projection, or tensors of their own."""
    n = h + hk * (2 if values else 1)
    x = _normal(gen, tokens, n + (hk if packed and not values else 0), dim).half()
    parts = [x[:, :h], x[:, h:h + hk], x[:, h + hk:h + 2 * hk]][:3 if values else 2]
    return [p if packed else p.contiguous() for p in parts]


def prepare(case, seed):
    gen = torch.Generator(device=_DEV).manual_seed(int(seed))
    s = dict(case=case)
    if case["op"] == "rotate":
        t = case["tokens"]
        _rotary(gen, s, case)
        s["q"], s["k"] = _heads(gen, t, case["heads"], case["kv_heads"], case["dim"], case["packed"], False)
        s["positions"] = torch.randint(0, 16384, (t,), generator=gen, device=_DEV, dtype=torch.int32)
        s["q_out"] = torch.empty((t, case["heads"], case["dim"]), dtype=torch.float16, device=_DEV)
        s["k_out"] = torch.empty((t, case["kv_heads"], case["dim"]), dtype=torch.float16, device=_DEV)
        return s
    q, ctx = _lengths(case)
    hk, dim, bs = case["kv_heads"], case["dim"], case["block"]
    s["tables"], blocks = _tables(gen, ctx, bs)
    s["ctx"], s["qlen"] = _ints(ctx), _ints(q)
    s["q_start"] = _ints([sum(q[:b]) for b in range(len(q))])
    total, s["max_q"], s["max_ctx"] = sum(q), max(q), max(ctx)
    if case["op"] == "tree" and case["bits"] == 16:
        s["key"] = _keys(gen, blocks, bs, hk, dim)
        s["value"] = _normal(gen, blocks, bs, hk, dim).half()
        s["key_exps"] = s["value_exps"] = None
    else:
        if case["op"] in ("read", "tree"):
            s["key"], s["key_exps"] = _quantise_blocks(_keys(gen, blocks, bs, hk, dim))
            s["value"], s["value_exps"] = _quantise_blocks(_normal(gen, blocks, bs, hk, dim).half())
        else:
            for name in ("key", "value"):
                s[name] = torch.zeros((blocks, bs, hk, dim), dtype=torch.float8_e4m3fn, device=_DEV)
                s[name + "_exps"] = torch.zeros((blocks, hk, bs), dtype=torch.uint8, device=_DEV)
    if case["op"] in ("write", "store"):
        s["starts"], s["out_starts"], rows = s["ctx"] - s["qlen"], s["q_start"], total
    elif case["op"] == "read":
        s["starts"] = torch.zeros_like(s["ctx"])
        s["out_starts"], rows = _ints([sum(ctx[:b]) for b in range(len(ctx))]), sum(ctx)
        s["max_q"] = s["max_ctx"]
    if case["op"] != "tree":
        s["k_out"] = torch.empty((rows, hk, dim), dtype=torch.float16, device=_DEV)
        s["v_out"] = torch.empty((rows, hk, dim), dtype=torch.float16, device=_DEV)
    if case["op"] == "write":
        s["k"] = _keys(gen, total, hk, dim)
        s["v"] = _normal(gen, total, hk, dim).half()
    elif case["op"] == "store":
        _rotary(gen, s, case)
        s["q"], s["k"], s["v"] = _heads(gen, total, case["heads"], hk, dim, True, True)
        s["positions"] = (s["starts"].repeat_interleave(s["qlen"].long())
                          + torch.arange(total, device=_DEV)
                          - s["q_start"].repeat_interleave(s["qlen"].long())).to(torch.int32)
        s["q_out"] = torch.empty((total, case["heads"], dim), dtype=torch.float16, device=_DEV)
    elif case["op"] == "tree":
        s["q"] = _normal(gen, total, case["heads"], dim).half()
        s["out"] = torch.empty_like(s["q"])
        s["parents"] = None if case["chain"] else _trees(seed, q)
    if own:
        import paged_kv_cache_206_gb300 as pa
        if case["op"] == "tree":
            s["step"] = pa.TreeStep(s["key"], s["value"], s["key_exps"], s["value_exps"], batch=len(q),
                                    num_heads=case["heads"], max_seqlen_q=s["max_q"],
                                    max_blocks_per_seq=s["tables"].shape[1])
        else:
            s["cache"] = pa.QuantCache(s["key"], s["value"], s["key_exps"], s["value_exps"])
    return s


def _trees(seed, q):
    """Parents of each sequence's drafts: mostly a recent token, some a root."""
    rng = random.Random(int(seed))
    return _ints([-1 if i == 0 or rng.random() < 0.1 else rng.randint(max(0, i - 6), i - 1)
                  for n in q for i in range(n)])


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


def _rows(s, start, count, width):
    """Sequences' positions start .. start + count, padded to `width`: which are there, and
    their blocks and places in them."""
    i = torch.arange(width, device=start.device)
    there = i < count[:, None]
    pos = torch.where(there, start[:, None] + i, torch.zeros_like(start)[:, None]).long()
    bs = s["key"].shape[1]
    return there, torch.gather(s["tables"].long(), 1, pos // bs), pos % bs


def _held(cache, exps, block, place):
    """The fp32 values that the cache holds at these places."""
    x = cache.view(torch.uint8)[block, place].view(torch.float8_e4m3fn).float() if exps is not None \
        else cache[block, place].float()
    return x if exps is None else torch.ldexp(x, exps.transpose(1, 2)[block, place].int()[..., None] - 127)


def _rotate(s, x, weight):
    case = s["case"]
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * weight.float()
    rot = case["rot"]
    c, z = s["cos_sin"][s["positions"].long()][:, None].split(rot // 2, -1)
    if case["interleaved"]:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack([a * c - b * z, b * c + a * z], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat([a * c - b * z, b * c + a * z], -1)
    return torch.cat([turned, y[..., rot:]], -1)


def _put(s, name, x):
    there, block, place = _rows(s, s["starts"], s["qlen"], s["max_q"])
    block, place = block[there], place[there]
    codes, e = _quantise(x)
    s[name].view(torch.uint8)[block, place] = codes.view(torch.uint8)
    s[name + "_exps"].transpose(1, 2)[block, place] = (e + 127).to(torch.uint8)


def _get(s, name):
    there, block, place = _rows(s, s["starts"], s["ctx"] - s["starts"], s["max_q"])
    return _held(s[name], s[name + "_exps"], block[there], place[there]).half()


def _tree(s):
    case, q = s["case"], s["q"]
    b, hk, width, longest = case["batch"], case["kv_heads"], s["max_q"], s["max_ctx"]
    zero = torch.zeros_like(s["ctx"])
    there, block, place = _rows(s, zero, s["ctx"], longest)
    k = _held(s["key"], s["key_exps"], block, place)
    v = _held(s["value"], s["value_exps"], block, place)
    live = torch.arange(width, device=q.device) < s["qlen"][:, None]
    rows = torch.zeros((b, width) + q.shape[1:], device=q.device)
    rows[live] = q.float()
    group = q.shape[1] // hk
    rows = rows.view(b, width, hk, group, -1).permute(0, 2, 1, 3, 4).flatten(2, 3)
    score = torch.matmul(rows, k.permute(0, 2, 3, 1)) / math.sqrt(case["dim"])
    # draft i sees draft j: itself and its ancestors, by doubling the steps taken
    i = torch.arange(width, device=q.device)
    if s["parents"] is None:
        sees = (i[:, None] >= i).expand(b, width, width)
    else:
        up = torch.full((b, width), -1, device=q.device, dtype=torch.int64)
        up[live] = s["parents"].long()
        step = (up[..., None] == i).float() + (i[:, None] == i).float()
        for _ in range(max(1, (width - 1).bit_length())):
            step = (torch.matmul(step, step) > 0).float()
        sees = step > 0
    pos = torch.arange(longest, device=q.device)
    draft = pos - (s["ctx"] - s["qlen"])[:, None]
    own_draft = torch.gather(sees, 2, draft.clamp(0, width - 1)[:, None].expand(b, width, longest))
    seen = there[:, None] & ((draft < 0)[:, None] | own_draft)
    seen = seen[:, None, :, None].expand(b, hk, width, group, longest).flatten(2, 3)
    score = torch.where(seen, score, torch.full_like(score, -math.inf))
    p = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-1e30))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    out = torch.matmul(p, v.permute(0, 2, 1, 3))
    out = out.view(b, hk, width, group, -1).permute(0, 2, 1, 3, 4).flatten(2, 3)
    return out[live].half()


def run(s):
    op, case = s["case"]["op"], s["case"]
    if own:
        import paged_kv_cache_206_gb300 as pa
        if op == "rotate":
            pa.pa_qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["cos_sin"], s["positions"],
                               s["q_out"], s["k_out"], eps=1e-6, interleaved=case["interleaved"])
            return s["q_out"], s["k_out"]
        if op == "tree":
            return s["step"].run(s["q"], s["tables"], s["ctx"], s["qlen"], s["parents"], s["out"])
        if op == "write":
            s["cache"].write(s["k"], s["v"], s["tables"], s["ctx"], s["qlen"], s["max_q"])
        elif op == "store":
            s["cache"].store(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["cos_sin"],
                             s["positions"], s["tables"], s["ctx"], s["qlen"], s["max_q"], s["q_out"],
                             eps=1e-6, interleaved=case["interleaved"])
        s["cache"].read(s["tables"], s["starts"], s["ctx"], s["out_starts"], s["max_q"], s["k_out"],
                        s["v_out"])
        return (s["k_out"], s["v_out"]) + ((s["q_out"],) if op == "store" else ())
    if op == "rotate":
        return _rotate(s, s["q"], s["q_weight"]).half(), _rotate(s, s["k"], s["k_weight"]).half()
    if op == "tree":
        return _tree(s)
    if op == "read":
        return _get(s, "key"), _get(s, "value")
    if op == "write":
        _put(s, "key", s["k"].float())
        _put(s, "value", s["v"].float())
        return _get(s, "key"), _get(s, "value")
    turned = _rotate(s, s["q"], s["q_weight"]).half()
    _put(s, "key", _rotate(s, s["k"], s["k_weight"]))
    _put(s, "value", s["v"].float())
    return _get(s, "key"), _get(s, "value"), turned


def work(case):
    dim = case["dim"]
    if case["op"] == "rotate":
        n = case["tokens"] * (case["heads"] + case["kv_heads"]) * dim
        return dict(bytes=n * 4 + case["tokens"] * (case["rot"] * 4 + 4), flops=n * 8)
    q, ctx = _lengths(case)
    hk = case["kv_heads"]
    if case["op"] == "read":
        n = sum(ctx) * hk * 2
        return dict(bytes=n * (dim * 3 + 1), flops=n * dim)
    if case["op"] in ("write", "store"):
        n = sum(q) * hk * 2  # read, written in 8 bits, and given back in 16
        b, f = n * (dim * 5 + 1), n * dim * 4
        if case["op"] == "store":
            m = sum(q) * case["heads"] * dim
            b, f = b + m * 4 + sum(q) * (case["rot"] * 4 + 4), f + m * 8 + n * dim * 4
        return dict(bytes=b, flops=f)
    row = case["dim"] * 2 if case["bits"] == 16 else case["dim"] + 1
    return dict(bytes=sum(ctx) * hk * 2 * row + sum(q) * case["heads"] * dim * 4,
                flops=4 * case["heads"] * dim * sum(a * b for a, b in zip(q, ctx)))


# ---- the definitions in 64 bits

def _exact_rows(x, weight, table, positions, rot, interleaved):
    y = x.double()
    if weight is not None:
        y = y / ((y ** 2).sum(-1, keepdim=True) / y.shape[-1] + 1e-6).sqrt() * weight.double()
    out = y.clone()
    t = table.double()[positions.long()]
    for i in range(rot // 2):
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c, z = t[:, i, None], t[:, rot // 2 + i, None]
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


def _exact_held(s, name, b, n):
    """The first n tokens of sequence b, [n, Hk, D]."""
    pos = torch.arange(n, device=s["ctx"].device)
    bs = s["key"].shape[1]
    block, place = s["tables"][b].long()[pos // bs], pos % bs
    if s[name + "_exps"] is None:
        return s[name][block, place].double()
    codes = s[name].view(torch.uint8)[block, place].view(torch.float8_e4m3fn).double()
    e = s[name + "_exps"][block, :, place].double() - 127
    return codes * torch.exp2(e)[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rotate", "store"):
        turn = lambda x, w: _exact_rows(x, w, s["cos_sin"], s["positions"], case["rot"],  # noqa: E731
                                        case["interleaved"])
        if case["op"] == "rotate":
            return turn(s["q"], s["q_weight"]), turn(s["k"], s["k_weight"])
        return _exact_8bit(turn(s["k"], s["k_weight"])), _exact_8bit(s["v"]), turn(s["q"], s["q_weight"])
    if case["op"] == "write":
        return _exact_8bit(s["k"]), _exact_8bit(s["v"])
    q, ctx = _lengths(case)
    if case["op"] == "read":
        return tuple(torch.cat([_exact_held(s, name, b, n) for b, n in enumerate(ctx)])
                     for name in ("key", "value"))
    if 4 * case["heads"] * case["dim"] * sum(a * b for a, b in zip(q, ctx)) > 1e12:
        return None
    outs, at = [], 0
    parents = None if s["parents"] is None else s["parents"].tolist()
    for b, (n, length) in enumerate(zip(q, ctx)):
        k, v = _exact_held(s, "key", b, length), _exact_held(s, "value", b, length)
        rows = s["q"][at:at + n].double()
        seen = torch.zeros((n, length), dtype=torch.bool)
        seen[:, :length - n] = True
        for i in range(n):
            j = i
            while j >= 0:
                seen[i, length - n + j] = True
                j = j - 1 if parents is None else parents[at + j]
        group = case["heads"] // case["kv_heads"]
        score = torch.einsum("nhgd,lhd->hgnl", rows.view(n, case["kv_heads"], group, -1), k)
        score = (score / case["dim"] ** 0.5).masked_fill(~seen.to(score.device), -math.inf)
        out = torch.einsum("hgnl,lhd->nhgd", torch.softmax(score, -1), v)
        outs.append(out.reshape(n, case["heads"], -1))
        at += n
    return torch.cat(outs)
