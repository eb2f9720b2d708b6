"""pa_tree_forward on the GPU against the 64-bit reference: trees, chains and
single tokens, over the fp16 and the 8-bit cache."""
import math

import numpy as np
import pytest

import paged_kv_cache_206_gb300 as pa
from . import serving_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    torch.cuda.set_device(0)
    return torch


def up(torch, a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Case:
    """A batch with its caches, on the host and on the GPU. Every cache slot
    that no sequence uses holds NaN (and exponent bytes of 255)."""

    def __init__(self, torch, bits, q, ctx, H, Hk, hk, hv, bs, kind, seed=0, sigma=1.0, behind=0,
                 scale=0.0, poison=None):
        rng = np.random.default_rng(seed + 13 * len(q) + hk)
        self.batch = batch = ref.make_batch(rng, q, ctx, bs)
        self.parents = ref.trees(rng, q, kind)
        T = int(batch.q.sum())
        self.tokens = T
        self.query = rng.normal(size=(T + behind, H, hk)).astype(np.float16)
        used = np.zeros((batch.num_blocks, bs), bool)
        for b in range(len(q)):
            used[batch.slots(b, 0, int(batch.ctx[b]))] = True
        self.dev, self.real, self.exp = [], [], []
        for hs in (hk, hv):
            x = (sigma * rng.normal(size=(batch.num_blocks, bs, Hk, hs))
                 * 2.0 ** rng.integers(-3, 2, (batch.num_blocks, bs, Hk, 1))).astype(np.float16)
            if poison:
                poison(self, x)
            if bits == 8:
                codes, e = ref.quantise(x.astype(np.float64))
                codes[~used], be = 0x7F, (e + 127).astype(np.uint8)
                be[~used] = 255
                self.real.append(ref.decode(codes) * 2.0 ** e[..., None].astype(np.float64))
                self.exp.append(np.swapaxes(e, 1, 2))
                self.dev.append((up(torch, codes).view(torch.float8_e4m3fn),
                                 up(torch, np.swapaxes(be, 1, 2))))
            else:
                x[~used] = np.nan
                self.real.append(x.astype(np.float64))
                self.exp.append(np.zeros((batch.num_blocks, Hk, bs)))
                self.dev.append((up(torch, x), None))
        self.scale = scale if scale > 0 else 1 / math.sqrt(hk)
        (k, ke), (v, ve) = self.dev
        self.step = pa.TreeStep(k, v, ke, ve, batch=len(q), num_heads=H, max_seqlen_q=max(max(q), 1),
                                max_blocks_per_seq=batch.tables.shape[1], scale=scale)
        par = None if self.parents is None else np.concatenate([self.parents, np.full(behind, 99, np.int32)])
        self.args = [up(torch, a) for a in (self.query, batch.tables, batch.ctx, batch.q, par)]
        self.out = torch.full((T + behind, H, hv), 7.0, dtype=torch.float16, device="cuda")

    def run(self, stream=None):
        return self.step.run(*self.args, self.out, stream=stream)

    def check(self, rows=slice(None)):
        want, bound = ref.tree_attention(self.query[:self.tokens], *self.real, *self.exp, self.batch,
                                         self.parents, self.scale)
        got = self.out.cpu().numpy().astype(np.float64)
        assert (got[self.tokens:] == 7).all()  # rows behind the last sequence
        got, want, bound = got[:self.tokens][rows], want[rows], bound[rows]
        err = np.abs(got - want)
        assert np.isfinite(got).all()
        assert (err <= bound).all(), (float((err / bound).max()), np.argwhere(err > bound)[:4])


# q, ctx, H, Hk, hk, hv, block, kind
CASES = [
    ([1], [1], 1, 1, 64, 64, 16, "chain"),
    ([1], [1], 32, 8, 128, 128, 128, "tree"),
    ([1, 1, 1], [15, 16, 17], 8, 2, 128, 128, 16, "chain"),
    ([1, 1], [1000, 333], 32, 8, 128, 128, 64, "chain"),
    ([4, 4], [4, 517], 4, 4, 128, 128, 128, "chain"),
    ([5, 0, 16, 1], [5, 40, 100, 77], 8, 2, 64, 64, 48, "tree"),
    ([16, 3], [300, 64], 32, 8, 128, 128, 32, "tree"),
    ([7], [200], 6, 3, 256, 256, 64, "tree"),
    ([2, 9], [70, 31], 16, 1, 256, 256, 16, "star"),
    ([64], [64], 8, 2, 128, 128, 64, "tree"),
    ([64, 17], [700, 90], 8, 2, 128, 128, 128, "line"),
    ([33], [2100], 4, 4, 64, 64, 128, "roots"),
    ([256], [300], 2, 2, 64, 64, 64, "tree"),
    ([100, 256], [100, 1000], 4, 1, 128, 128, 128, "tree"),
    ([300], [400], 4, 2, 128, 128, 128, "chain"),
    ([3, 2], [40, 9], 4, 2, 48, 80, 16, "tree"),
    ([2], [50], 3, 1, 576, 512, 32, "tree"),
    ([1] * 70, list(range(1, 71)), 4, 2, 64, 64, 16, "chain"),
    ([8] * 3, [5000, 8, 2500], 28, 4, 128, 128, 128, "tree"),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("bits", [8, 16])
def test_tree(torch, bits, case):
    c = Case(torch, bits, *case, behind=2)
    c.run()
    assert c.step.status() == (pa.PA_OK, 0)
    c.check()


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("sigma", [2.0**-9, 30.0])
def test_small_and_large_values(torch, bits, sigma):
    c = Case(torch, bits, [6, 1], [90, 200], 8, 2, 128, 128, 16, "tree", sigma=sigma, scale=0.01)
    c.run()
    c.check()


def test_line_is_a_chain(torch):
    """A tree whose every draft follows the one before is the chain, bit for bit."""
    a = Case(torch, 8, [20, 7], [400, 7], 8, 2, 128, 128, 64, "line")
    a.run()
    got = a.out.clone()
    a.args[4] = None
    a.run()
    assert torch.equal(got, a.out)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("shape", [(2, 2, 64, 64), (8, 2, 128, 128), (16, 1, 128, 128), (4, 1, 256, 256),
                                   (2, 1, 48, 32)], ids=str)
@pytest.mark.parametrize("bad", ["key", "value"])
def test_drafts_that_a_row_does_not_see_do_not_touch_it(torch, bits, shape, bad):
    """NaN and infinities in one draft's key or value reach exactly the rows
    that have it among their ancestors."""
    H, Hk, hk, hv = shape
    q, ctx = [9, 12], [50, 12]
    hit = [(0, 4), (1, 0), (1, 7)]  # (sequence, draft)

    def poison(case, x):
        which = len(case.real)  # 0 while the keys are made, 1 for the values
        if (which == 0) != (bad == "key"):
            return
        for n, (b, i) in enumerate(hit):
            blk, off = case.batch.slots(b, ctx[b] - q[b] + i, ctx[b] - q[b] + i + 1)
            x[blk[0], off[0], :, n % 3] = [np.nan, np.inf, -np.inf][n % 3]

    c = Case(torch, bits, q, ctx, H, Hk, hk, hv, 16, "tree", poison=poison)
    c.run()
    got = c.out.cpu().numpy()
    touched = np.zeros(len(got), bool)
    for b, i in hit:
        t0 = int(c.batch.starts[b])
        m = ref.sees(q[b], c.parents[t0:t0 + q[b]])
        touched[t0:t0 + q[b]] |= m[:, i]
    assert touched.any() and not touched.all()
    assert np.isfinite(got[~touched]).all()
    broken = ~np.isfinite(got[touched]).all(axis=(1, 2))
    if bad == "value":
        assert broken.all()
    # the rows that do not see it are what they are without it
    clean = Case(torch, bits, q, ctx, H, Hk, hk, hv, 16, "tree")
    clean.run()
    want, bound = ref.tree_attention(clean.query, *clean.real, *clean.exp, clean.batch, clean.parents,
                                     clean.scale)
    err = np.abs(got.astype(np.float64) - want)
    assert (err[~touched] <= bound[~touched]).all()


def test_bad_parents_lengths_and_blocks(torch):
    c = Case(torch, 8, [4, 3], [40, 30], 8, 2, 128, 128, 16, "tree")
    par = c.parents.copy()
    par[2], par[5] = 2, -7  # a draft that follows itself, and no draft at all: both roots
    c.args[4] = up(torch, par)
    c.run()
    st, bits = c.step.status()
    assert st == pa.PA_ERR_INVALID_ARG and bits == pa.PA_STATUS_BIT_TREE
    par[2] = par[5] = -1
    c.parents = par
    c.check()
    pa.pa_status_clear(c.step.workspace)
    c = Case(torch, 8, [4, 3], [40, 30], 8, 2, 128, 128, 16, "tree")
    ctx = c.batch.ctx.copy()
    ctx[0] = 3
    c.args[2] = up(torch, ctx)
    c.run()
    assert c.step.status() == (pa.PA_ERR_INVALID_ARG, pa.PA_STATUS_BIT_PLAN)
    # the other sequence is right (the keys are split where the batch's lengths
    # put it, so not bit for bit what it is in another batch)
    assert (c.out[:4] == 7).all()
    c.check(slice(4, 7))
    c = Case(torch, 8, [4, 3], [40, 30], 8, 2, 128, 128, 16, "tree")
    tables = c.batch.tables.copy()
    tables[0, 1] = c.batch.num_blocks
    c.args[1] = up(torch, tables)
    c.run()
    assert c.step.status() == (pa.PA_ERR_BLOCK_INDEX, pa.PA_STATUS_BIT_BLOCK_INDEX)
    c.check(slice(4, 7))


def test_captured_and_replayed_with_other_lengths(torch):
    c = Case(torch, 8, [8, 8], [900, 900], 32, 8, 128, 128, 64, "tree")
    s = torch.cuda.Stream()
    c.run(stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.run()
    g.replay()
    torch.cuda.synchronize()
    c.check()
    # shorter contexts: the same blocks, whose first tokens are all there
    c.batch.ctx[:] = [333, 8]
    c.args[2].copy_(up(torch, c.batch.ctx))
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    c.check()


def test_one_step_of_speculation(torch):
    """Store a prompt, then store a tree of drafts and attend it over the cache;
    the prompt read back feeds the fp16 forward pass with the same result."""
    rng = np.random.default_rng(11)
    H, Hk, d, bs = 8, 2, 128, 16
    ctx, q = np.array([37, 80], np.int32), np.array([6, 9], np.int32)
    batch = ref.make_batch(rng, q, ctx + q, bs)
    parents = ref.trees(rng, q, "tree")
    cos = np.arange(200)[:, None] * 10000.0 ** (-np.arange(0, d, 2) / d)
    table = up(torch, np.concatenate([np.cos(cos), np.sin(cos)], 1).astype(np.float32))
    w = up(torch, (1 + 0.1 * rng.normal(size=d)).astype(np.float16))
    cache = pa.QuantCache.empty(batch.num_blocks, bs, Hk, d)
    tables = up(torch, batch.tables)

    def project(n):
        x = up(torch, rng.normal(size=(n, H + 2 * Hk, d)).astype(np.float16))
        return x[:, :H], x[:, H:H + Hk], x[:, H + Hk:]

    T = int(ctx.sum())
    qo = torch.empty((T, H, d), dtype=torch.float16, device="cuda")
    cache.store(*project(T), w, w, table, None, tables, up(torch, ctx), up(torch, ctx), int(ctx.max()), qo)
    # the drafts' positions: the prompt's length plus their depth
    depth = np.zeros(len(parents), np.int32)
    for b in range(2):
        t0 = int(batch.starts[b])
        for i in range(q[b]):
            p = parents[t0 + i]
            depth[t0 + i] = ctx[b] if p < 0 else depth[t0 + p] + 1
    n = int(q.sum())
    qd = torch.empty((n, H, d), dtype=torch.float16, device="cuda")
    cache.store(*project(n), w, w, table, up(torch, depth), tables, up(torch, ctx + q), up(torch, q),
                int(q.max()), qd)
    step = pa.TreeStep(cache.key, cache.value, cache.key_exps, cache.value_exps, batch=2, num_heads=H,
                       max_seqlen_q=int(q.max()), max_blocks_per_seq=batch.tables.shape[1])
    out = torch.empty((n, H, d), dtype=torch.float16, device="cuda")
    step.run(qd, tables, up(torch, ctx + q), up(torch, q), up(torch, parents), out)
    assert step.status() == (pa.PA_OK, 0)
    # read back into an fp16 paged cache of its own blocks
    need = -(-(ctx + q) // bs)
    first = (np.cumsum(need) - need).astype(np.int32)
    k16 = torch.zeros((int(need.sum()), bs, Hk, d), dtype=torch.float16, device="cuda")
    v16 = torch.zeros_like(k16)
    cache.read(tables, None, up(torch, ctx + q), up(torch, first * bs), int((ctx + q).max()),
               k16.view(-1, Hk, d), v16.view(-1, Hk, d))
    own = np.zeros((2, int(need.max())), np.int32)
    for b in range(2):
        own[b, :need[b]] = first[b] + np.arange(need[b])
    half = pa.TreeStep(k16, v16, batch=2, num_heads=H, max_seqlen_q=int(q.max()),
                       max_blocks_per_seq=own.shape[1])
    out16 = torch.empty_like(out)
    half.run(qd, up(torch, own), up(torch, ctx + q), up(torch, q), up(torch, parents), out16)
    real = [t.double().cpu().numpy() for t in (k16, v16)]
    nowhere = np.zeros((len(k16), Hk, bs))
    flat = ref.Batch(own, ctx + q, q, bs, len(k16))
    want, bound = ref.tree_attention(qd.cpu().numpy(), *real, nowhere, nowhere, flat, parents,
                                     1 / math.sqrt(d))
    # (the bound of the 8-bit cache is the larger one: weights relative to the largest p 2^ev)
    ev = cache.value_exps.cpu().numpy().astype(np.float64) - 127
    ev_own = np.zeros_like(nowhere)
    for b in range(2):
        ev_own[own[b, :need[b]]] = ev[batch.tables[b, :need[b]]]
    _, wide = ref.tree_attention(qd.cpu().numpy(), *real, nowhere, ev_own, flat, parents, 1 / math.sqrt(d))
    for got, limit in ((out16, bound), (out, np.maximum(bound, wide))):
        assert (np.abs(got.cpu().numpy() - want) <= limit).all()
    # the plain forward pass of the framework, on single tokens over the same cache
    cfg = pa.make_config(batch=2, num_heads=H, kv_heads=Hk, head_size_k=d, block_size=bs,
                         num_blocks=len(k16), max_blocks_per_seq=own.shape[1], num_sms=8)
    plan = pa.pa_plan(cfg, ctx)
    q1 = qo[[int(ctx[0]) - 1, T - 1]].contiguous()
    a, b = torch.empty_like(q1), torch.empty_like(q1)
    ws = torch.zeros(max(plan.workspace_bytes, 256), dtype=torch.uint8, device="cuda")
    comb = up(torch, plan.combine) if len(plan.combine) else None
    pa.pa_forward(cfg, q1, k16, v16, up(torch, own), up(torch, ctx), None, None, None, up(torch, plan.work),
                  comb, ws, a)
    one = pa.TreeStep(k16, v16, batch=2, num_heads=H, max_seqlen_q=1, max_blocks_per_seq=own.shape[1])
    one.run(q1, up(torch, own), up(torch, ctx), None, None, b)
    flat = ref.Batch(own, ctx, np.ones(2, np.int32), bs, len(k16))
    want, bound = ref.tree_attention(q1.cpu().numpy(), *real, nowhere, nowhere, flat, None,
                                     1 / math.sqrt(d))
    # pa_forward rounds each split's partial row to fp16 as well: 2^-11 of the magnitudes
    mags, _ = ref.tree_attention(q1.cpu().numpy(), real[0], np.abs(real[1]), nowhere, nowhere, flat, None,
                                 1 / math.sqrt(d))
    assert (np.abs(b.cpu().numpy() - want) <= bound).all()
    assert (np.abs(a.cpu().numpy() - want) <= bound + 2.0**-11 * mags).all()


@pytest.mark.parametrize("bits,drafts", [(8, 16), (8, 64), (16, 64), (8, 4)])
def test_long_contexts_again_and_again(torch, bits, drafts):
    """Full batches of long contexts, where copies land in any order: every run of
    three states in turn gives the state's first bits, and the first sequence is
    attention in 64 bits. Tolerance: weights and outputs are rounded to fp16 (2^-11
    each, relative to sum p |v|); the fp32 scores are off by at most
    128 * 2^-24 * 82 * 0.09 = 6e-5 of a weight, well within the tenth on top."""
    B, H, Hk, d, bs = 24, 32, 8, 128, 128
    rng = np.random.default_rng(drafts)
    states = []
    for n in range(3):
        g = torch.Generator(device="cuda").manual_seed(100 * drafts + n)
        q = rng.integers(max(1, drafts // 2), drafts + 1, B).astype(np.int32)
        ctx = np.maximum(q, rng.integers(64, 8193, B)).astype(np.int32)
        need = -(-ctx // bs)
        ids = rng.permutation(int(need.sum())).astype(np.int32)
        tables = np.full((B, int(need.max())), -1, np.int32)
        for b in range(B):
            tables[b, :need[b]] = ids[need[:b].sum():need[:b + 1].sum()]
        parents = ref.trees(rng, q, "tree")
        k, v = (torch.randn((len(ids), bs, Hk, d), generator=g, device="cuda").half() for _ in range(2))
        exps = [None, None]
        if bits == 8:
            k, v = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)
            exps = [torch.randint(125, 129, (len(ids), Hk, bs), generator=g, device="cuda").to(torch.uint8)
                    for _ in range(2)]
        query = torch.randn((int(q.sum()), H, d), generator=g, device="cuda").half()
        step = pa.TreeStep(k, v, *exps, batch=B, num_heads=H, max_seqlen_q=drafts,
                           max_blocks_per_seq=tables.shape[1])
        args = query, up(torch, tables), up(torch, ctx), up(torch, q), up(torch, parents)
        states.append((step, args, torch.empty_like(query), k, v, exps, q, ctx, tables, parents))
    torch.cuda.synchronize()
    first = []
    for step, args, out, k, v, exps, q, ctx, tables, parents in states:
        first.append(step.run(*args, out).clone())
        L, n = int(ctx[0]), int(q[0])
        rows = torch.from_numpy(tables[0, :-(-L // bs)].astype(np.int64)).cuda()
        keys, vals = (t[rows].double() for t in (k, v))
        if bits == 8:
            keys, vals = (t * (2.0 ** (e[rows].double() - 127)).transpose(1, 2)[..., None]
                          for t, e in zip((keys, vals), exps))
        keys, vals = (t.reshape(-1, Hk, d)[:L].repeat_interleave(H // Hk, 1) for t in (keys, vals))
        see = np.zeros((n, L), bool)
        see[:, :L - n] = True
        for i in range(n):
            a = i
            while a >= 0:
                see[i, L - n + a] = True
                a = int(parents[a])
        s = torch.einsum("qhd,khd->hqk", args[0][:n].double(), keys) / math.sqrt(d)
        p = s.masked_fill(~torch.from_numpy(see).cuda(), -math.inf).softmax(-1)
        want, size = (torch.einsum("hqk,khd->qhd", p, t) for t in (vals, vals.abs()))
        assert ((first[-1][:n].double() - want).abs() <= 1.1 * 2.0**-10 * size + 1e-7).all()
    for i in range(45):
        step, args, out = states[i % 3][:3]
        assert torch.equal(step.run(*args, out), first[i % 3]), i


def speculation(torch, seed, bs=32, drafts=5):
    """Inputs of a step: store the drafts into an 8-bit cache, then attend them."""
    B, H, Hk, d = 6, 8, 2, 128
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    q = rng.integers(1, drafts + 1, B).astype(np.int32)
    ctx = (q + rng.integers(1, 700, B)).astype(np.int32)
    cols = int(-(-ctx.max() // bs))
    T = int(q.sum())
    cache = pa.QuantCache.empty(B * cols, bs, Hk, d)
    old = [torch.randn((int(ctx.sum()), Hk, d), generator=g, device="cuda").half() for _ in range(2)]
    tables = up(torch, np.arange(B * cols, dtype=np.int32).reshape(B, cols))
    cache.write(*old, tables, up(torch, ctx), up(torch, ctx), int(ctx.max()))
    x = torch.randn((T, H + 2 * Hk, d), generator=g, device="cuda").half()
    cs = torch.randn((2048, d), generator=g, device="cuda")
    step = pa.TreeStep(cache.key, cache.value, cache.key_exps, cache.value_exps, batch=B, num_heads=H,
                       max_seqlen_q=drafts, max_blocks_per_seq=cols)
    qr, out = (torch.empty((T, H, d), dtype=torch.float16, device="cuda") for _ in range(2))
    lens, qlens, parents = up(torch, ctx), up(torch, q), up(torch, ref.trees(rng, q, "tree"))

    def run(stream=None):
        cache.store(x[:, :H], x[:, H:H + Hk], x[:, H + Hk:], None, None, cs, None, tables, lens, qlens,
                    drafts, qr, stream=stream)
        step.run(qr, tables, lens, qlens, parents, out, stream=stream)
        return out
    run.x = x
    torch.cuda.synchronize()
    return run


def test_two_streams_at_once(torch):
    """Two steps with a workspace each, at work side by side on streams of their own,
    give what they give alone."""
    runs = [speculation(torch, s) for s in (1, 2)]
    alone = [r().clone() for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    for _ in range(25):
        for r, s in zip(runs, streams):
            got = r(stream=s)
    torch.cuda.synchronize()
    for r, want in zip(runs, alone):
        with torch.cuda.stream(streams[0]):
            got = r()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_store_and_tree_captured_and_replayed(torch):
    """A captured step replayed on other queries, keys and values, next to the same
    step run eagerly."""
    run, s = speculation(torch, 3), torch.cuda.Stream()
    with torch.cuda.stream(s):
        run()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = run()
        for n in range(3):
            run.x.copy_(torch.randn(run.x.shape, device="cuda").half())
            g.replay()
            s.synchronize()
            got = out.clone()
            out.fill_(0)
            want = run().clone()
            s.synchronize()
            assert torch.equal(got, want) and bool(got.isfinite().all()), n


@pytest.mark.parametrize("sizes", [(16, 16), (32, 48), (80, 80), (96, 96), (112, 64), (64, 112), (144, 144),
                                   (192, 128), (240, 256), (272, 256)], ids=str)
@pytest.mark.parametrize("bits", [8, 16])
def test_head_sizes_between_the_tiles(torch, bits, sizes):
    """Heads that fill no tile's dims, unlike ones, in tiles of 8 and 16 rows and several of them;
    what lies next to a head's row (its neighbours' rows and NaN) does not reach it."""
    for q, ctx, H, Hk, bs in (([1, 1, 1], [1, 33, 700], 8, 2, 16), ([5, 0, 3], [90, 40, 1300], 6, 3, 48),
                              ([13], [777], 12, 3, 128)):
        c = Case(torch, bits, q, ctx, H, Hk, *sizes, bs, "tree", behind=1)
        c.run()
        c.check()
        assert c.step.status() == (pa.PA_OK, 0)


@pytest.mark.parametrize("drafts,lo,hi", [(16, 0, 300), (5, 0, 40), (64, 100, 700)])
def test_many_ends_of_contexts_in_turn(torch, drafts, lo, hi):
    """Hundreds of short contexts, so that a stage whose rows behind the context were cleared (they
    hold NaN, and some drafts' values do) is filled again at once: every run gives the same bits, and
    the rows of every tenth sequence that see no NaN are attention in 64 bits."""
    rng = np.random.default_rng(drafts)
    B = 200
    q = rng.integers(max(1, drafts // 2), drafts + 1, B)
    ctx = q + rng.integers(lo, hi, B)
    nan = []

    def poison(case, x):
        if len(case.real) == 0:
            return
        for b in range(0, B, 3):
            i = int(q[b]) - 1  # the last draft, which none but itself sees
            blk, off = case.batch.slots(b, int(ctx[b]) - 1, int(ctx[b]))
            x[blk[0], off[0], :, 5] = np.nan
            nan.append(int(case.batch.starts[b]) + i)

    c = Case(torch, 8, q, ctx, 32, 2, 128, 128, 16, "tree", poison=poison)
    c.run()
    first = c.out.clone()
    assert c.step.status() == (pa.PA_OK, 0)
    for _ in range(20):
        assert torch.equal(c.run().view(torch.int16), first.view(torch.int16))
    got = c.out.cpu().numpy()
    assert np.isnan(got[nan][:, :, 5]).all()
    some = ref.Batch(c.batch.tables[::10], c.batch.ctx[::10], c.batch.q[::10], 16, c.batch.num_blocks)
    at = np.concatenate([t + np.arange(n) for t, n in zip(c.batch.starts[::10], some.q)])
    for v in c.real:
        v[np.isnan(v)] = 0  # behind the contexts, and the drafts that only `nan` sees
    want, bound = ref.tree_attention(c.query[at], *c.real, *c.exp, some, c.parents[at], c.scale)
    ok = ~np.isin(at, nan)
    assert ok.any() and (np.abs(got[at].astype(np.float64) - want)[ok] <= bound[ok]).all()


@pytest.mark.parametrize("bits,H,drafts,lo,hi,d", [
    (8, 32, 64, 100, 700, 128), (8, 32, 8, 100, 700, 128), (8, 16, 32, 600, 1400, 128), (16, 32, 64, 100, 700, 128),
    (8, 8, 4, 100, 700, 128), (16, 8, 4, 100, 700, 128), (8, 8, 1, 1, 900, 128), (8, 8, 4, 50, 300, 64),
    (16, 8, 2, 50, 300, 64), (8, 8, 4, 50, 300, 256), (16, 8, 2, 50, 300, 256), (8, 12, 5, 50, 300, 96)])
def test_many_row_tiles_again_and_again(torch, bits, H, drafts, lo, hi, d):
    """Rings that never run empty while row tiles end, so that every stage is filled again as soon as
    it is given back: three hundred runs give the same bits."""
    rng = np.random.default_rng(drafts + H)
    q = rng.integers(max(1, drafts // 2), drafts + 1, 200)
    c = Case(torch, bits, q, q + rng.integers(lo, hi, 200), H, 2, d, d, 16, "tree")
    first = c.run().clone().view(torch.int16)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(300):
        differ += (c.run().view(torch.int16) != first).any()
    assert differ.item() == 0
    assert c.step.status() == (pa.PA_OK, 0)


# rows of a kv head: the kernels of up to 16, of up to 128 and of more; heads above 256 dims
UNWRITTEN = [(8, 2, 64, 2), (16, 2, 128, 1), (16, 1, 128, 8), (16, 1, 64, 20), (4, 2, 272, 3)]


@pytest.mark.parametrize("shape", UNWRITTEN, ids=str)
def test_an_empty_cache_gives_zeros(torch, shape):
    """A warm-up over a cache that nothing was written into."""
    H, Hk, d, q = shape
    c = Case(torch, 8, [q, 1], [300, 1], H, Hk, d, d, 16, "tree")
    e = pa.QuantCache.empty(c.batch.num_blocks, 16, Hk, d)
    c.step = pa.TreeStep(e.key, e.value, e.key_exps, e.value_exps, batch=2, num_heads=H, max_seqlen_q=q,
                         max_blocks_per_seq=c.batch.tables.shape[1])
    c.run()
    assert c.step.status() == (pa.PA_OK, 0) and bool((c.out == 0).all())


@pytest.mark.parametrize("shape", UNWRITTEN, ids=str)
@pytest.mark.parametrize("scale", [0.0, 1e-30])
def test_slots_that_were_never_written_are_zero_rows(torch, shape, scale):
    """Zero codes under zero exponent bytes amid a context, in all of a key tile, in all of a
    sequence, and in the values alone: keys of score 0 and values of 0."""
    H, Hk, d, q = shape
    c = Case(torch, 8, [q, q, 1, q], [400, 290, 9, 140 + q], H, Hk, d, d, 16, "tree", scale=scale)
    for n, (codes, exps) in enumerate(c.dev):
        for b, lo, hi in ((0, 3, 90), (0, 200, 201), (1, 0, 140), (2, 0, 9), (3, 20, 140 + q)):
            if (b, n) == (3, 0):
                continue
            blk, off = c.batch.slots(b, lo, hi)
            codes.view(torch.uint8)[blk, off] = 0
            exps.transpose(1, 2)[blk, off] = 0
            c.real[n][blk, off] = 0
            c.exp[n].transpose(0, 2, 1)[blk, off] = -127
    c.run()
    assert c.step.status() == (pa.PA_OK, 0)
    c.check()


# q, ctx, H, Hk, dims, block, kind: few rows of a kv head, up to 128, more; heads above 256 dims
SPREAD = [
    ([3, 2], [290, 40], 8, 2, 128, 16, "tree"),
    ([9, 12], [50, 300], 16, 2, 128, 16, "tree"),
    ([20, 7, 1], [150, 263, 128], 8, 4, 64, 48, "tree"),
    ([12], [520], 8, 1, 128, 64, "chain"),
    ([30, 9], [31, 400], 16, 2, 128, 32, "tree"),
    ([200], [700], 2, 1, 64, 128, "chain"),
    ([5], [200], 4, 2, 272, 16, "tree"),
]


@pytest.mark.parametrize("case", SPREAD, ids=str)
@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("big", ["key", "value", "both"])
def test_large_drafts_that_a_row_does_not_see_take_nothing_from_it(torch, bits, case, big):
    """One draft's key or value is of fp16's largest size among small ones: the rows that do not
    attend it are as exact as without it."""
    q, ctx, H, Hk, d, bs, kind = case

    def poison(case, x):
        which = ("key", "value")[len(case.real)]
        if which == "value":
            x *= np.float16(2.0**-9)
        if big not in (which, "both"):
            return
        for b, n in enumerate(q):
            blk, off = case.batch.slots(b, ctx[b] - n + n // 2, ctx[b] - n + n // 2 + 1)
            x[blk[0], off[0]] = np.where(x[blk[0], off[0]] < 0, -65504, 65504)

    c = Case(torch, bits, q, ctx, H, Hk, d, d, bs, kind, poison=poison)
    c.run()
    assert c.step.status() == (pa.PA_OK, 0)
    seen = np.zeros(c.tokens, bool)  # the rows that do attend it: their scores are no fp32 sums to bound
    for b, n in enumerate(q):
        t0 = int(c.batch.starts[b])
        seen[t0:t0 + n] = ref.sees(n, None if c.parents is None else c.parents[t0:t0 + n])[:, n // 2]
    if max(q) > 2:
        assert not seen.all()
    c.check(slice(None) if big == "value" else ~seen)


@pytest.mark.parametrize("case", SPREAD, ids=str)
@pytest.mark.parametrize("spread", [(0, 7), (0, 8), (0, 14), (0, 15), (-14, 13), (-24, 16)], ids=str)
@pytest.mark.parametrize("which", ["key", "value", "both"])
def test_rows_of_many_magnitudes_in_a_key_tile(torch, case, spread, which):
    """Exponents as far apart as a key tile's common one reaches, one further, and as far as
    fp16 goes, with zero rows among the widest."""
    q, ctx, H, Hk, d, bs, kind = case
    lo, hi = spread

    def poison(case, x):
        if which not in (("key", "value")[len(case.real)], "both"):
            return
        rng = np.random.default_rng(99)
        e = rng.integers(lo, hi, x.shape[:3] + (1,))
        x[:] = (rng.uniform(0.5, 0.99, x.shape) * 2.0**e * rng.choice([-1, 1], x.shape)).astype(np.float16)
        if lo < -20:
            x[rng.random(x.shape[:3]) < 0.1] = 0

    c = Case(torch, 8, q, ctx, H, Hk, d, d, bs, kind, poison=poison, scale=2.0 ** -(hi + 3))
    c.run()
    assert c.step.status() == (pa.PA_OK, 0)
    c.check()
