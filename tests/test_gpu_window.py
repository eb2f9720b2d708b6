"""pa_window_forward on the GPU against the 64-bit reference: decode steps, drafts, prompts and
parts of prompts, over the fp16 and the 8-bit cache."""
import math

import numpy as np
import pytest

import paged_kv_cache_206_gb300 as pa
from . import serving_ref as ref
from . import window_ref as wref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    torch.cuda.set_device(0)
    return torch


def up(torch, a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Case:
    """A batch with its caches, on the host and on the GPU. Every cache slot that no token attends
    holds NaN (and exponent bytes of 255), every table entry of a block without one that is
    attended -1 or anything."""

    def __init__(self, torch, bits, q, ctx, H, Hk, hk, hv, bs, window, sinks, seed=0, sigma=1.0, behind=0, scale=0.0,
                 poison=None, spread=(-3, 2), max_q=None):
        rng = np.random.default_rng(seed + 13 * len(q) + hk)
        self.window, self.sinks = window, sinks
        self.batch = batch = ref.make_batch(rng, q, ctx, bs)
        T = self.tokens = int(batch.q.sum())
        self.query = rng.normal(size=(T + behind, H, hk)).astype(np.float16)
        used = np.zeros((batch.num_blocks, bs), bool)
        tables = batch.tables.copy()
        for b in range(len(q)):
            n, L = int(batch.q[b]), int(batch.ctx[b])
            keys = np.flatnonzero(wref.sees(n, L, window, sinks).any(0)) if n else np.zeros(0, int)
            used[batch.tables[b, keys // bs], keys % bs] = True
            pages = np.setdiff1d(np.arange(tables.shape[1]), keys // bs)
            tables[b, pages] = rng.choice([-1, 2**31 - 1, 0, batch.num_blocks], len(pages))
        self.dev, self.real, self.exp = [], [], []
        for hs in (hk, hv):
            size = rng.normal if spread == (-3, 2) else lambda size: rng.uniform(0.5, 0.99, size)
            x = (sigma * size(size=(batch.num_blocks, bs, Hk, hs)) * rng.choice([-1, 1], (1, 1, 1, hs))
                 * 2.0 ** rng.integers(*spread, (batch.num_blocks, bs, Hk, 1))).astype(np.float16)
            if poison:
                poison(self, x)
            if bits == 8:
                codes, e = ref.quantise(x.astype(np.float64))
                codes[~used], be = 0x7F, (e + 127).astype(np.uint8)
                be[~used] = 255
                self.real.append(ref.decode(codes) * 2.0 ** e[..., None].astype(np.float64))
                self.exp.append(np.swapaxes(e, 1, 2))
                self.dev.append((up(torch, codes).view(torch.float8_e4m3fn), up(torch, np.swapaxes(be, 1, 2))))
            else:
                x[~used] = np.nan
                self.real.append(x.astype(np.float64))
                self.exp.append(np.zeros((batch.num_blocks, Hk, bs)))
                self.dev.append((up(torch, x), None))
        self.scale = scale if scale > 0 else 1 / math.sqrt(hk)
        (k, ke), (v, ve) = self.dev
        self.step = pa.WindowStep(k, v, ke, ve, batch=len(q), num_heads=H, max_seqlen_q=max_q or max(max(q), 1),
                                  max_blocks_per_seq=tables.shape[1], window=window, sinks=sinks, scale=scale)
        self.args = [up(torch, a) for a in (self.query, tables, batch.ctx, batch.q)]
        self.out = torch.full((T + behind, H, hv), 7.0, dtype=torch.float16, device="cuda")

    def run(self, stream=None):
        return self.step.run(*self.args, self.out, stream=stream)

    def want(self, only=None):
        return wref.window_attention(self.query[:self.tokens], *self.real, self.exp[1], self.batch, self.window,
                                     self.sinks, self.scale, only)

    def check(self, only=None):
        want, bound = self.want(only)
        got = self.out.cpu().numpy().astype(np.float64)
        assert (got[self.tokens:] == 7).all()  # rows behind the last sequence
        got = got[:self.tokens]
        if only is not None:
            rows = np.concatenate([self.batch.starts[b] + np.arange(self.batch.q[b]) for b in only])
            got, want, bound = got[rows], want[rows], bound[rows]
        assert np.isfinite(got).all()
        err = np.abs(got - want)
        assert (err <= bound).all(), (float((err / bound).max()), np.argwhere(err > bound)[:4])


# q, ctx, H, Hk, hk, hv, block, window, sinks
CASES = [
    ([1], [1], 1, 1, 64, 64, 16, 1, 0),
    ([1], [1], 32, 8, 128, 128, 128, 4, 4),
    ([1, 1, 1, 1], [15, 16, 17, 400], 8, 2, 128, 128, 16, 16, 0),
    ([1, 1, 1], [1000, 333, 40], 32, 8, 128, 128, 64, 100, 4),
    ([1, 1], [700, 90], 8, 8, 64, 64, 128, 1, 1),
    ([1, 1], [3000, 1025], 16, 1, 128, 128, 128, 1024, 130),
    ([1, 1], [900, 2000], 16, 1, 256, 256, 64, 300, 17),
    ([4, 4], [4, 517], 4, 4, 128, 128, 128, 33, 3),
    ([5, 0, 16, 1], [5, 40, 100, 777], 8, 2, 64, 64, 48, 50, 10),
    ([16, 3], [300, 64], 32, 8, 128, 128, 32, 2000, 0),
    ([7], [200], 6, 3, 256, 256, 64, 5, 64),
    ([2, 9], [70, 331], 16, 1, 256, 256, 16, 40, 5),
    ([9, 3, 1], [400, 3, 800], 12, 2, 96, 96, 16, 70, 20),
    ([3, 2], [40, 90], 4, 2, 48, 80, 16, 17, 2),
    ([2, 1], [500, 30], 3, 1, 576, 512, 32, 100, 40),
    ([1] * 70, list(range(1, 71)), 4, 2, 64, 64, 16, 20, 3),
    # more rows of a kv head: drafts, prompts, parts of prompts
    ([64], [64], 8, 2, 128, 128, 64, 20, 0),
    ([64, 17], [700, 90], 8, 2, 128, 128, 128, 200, 4),
    ([33], [2100], 4, 4, 64, 64, 128, 1000, 150),
    ([200], [200], 2, 2, 64, 64, 64, 64, 1),
    ([300, 5, 0, 129], [400, 700, 9, 129], 4, 2, 128, 128, 128, 128, 128),
    ([300], [300], 16, 2, 128, 128, 16, 100, 0),
    ([257, 1], [900, 1], 28, 4, 128, 128, 48, 300, 64),
    ([600, 100], [600, 1300], 6, 3, 64, 64, 32, 513, 7),
    ([500], [800], 1, 1, 128, 128, 128, 1, 0),
    ([500], [800], 1, 1, 64, 64, 16, 10**9, 10**9),
    ([400, 31], [450, 31], 5, 1, 128, 128, 64, 77, 2),
    ([130], [500], 40, 40, 64, 64, 128, 250, 4),
    ([40], [300], 64, 1, 128, 128, 64, 90, 33),
    ([20], [100], 160, 1, 64, 64, 16, 30, 3),
    ([9], [60], 300, 1, 128, 128, 16, 25, 3),
    ([50], [120], 40, 2, 256, 256, 16, 30, 5),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("bits", [8, 16])
def test_window(torch, bits, case):
    c = Case(torch, bits, *case, behind=2)
    c.run()
    assert c.step.status() == (pa.PA_OK, 0)
    c.check()


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("q,G", [(1, 4), (6, 4), (100, 1), (100, 4)], ids=str)
def test_every_border_of_a_window(torch, bits, q, G):
    """Windows and sinks that end on either side of a unit of keys, of a block and of a tile."""
    for window in (1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257):
        for sinks in (0, 1, 32, 128, 129):
            c = Case(torch, bits, [q, q], [q + 290, q], 2 * G, 2, 64, 64, 16 if window % 2 else 128, window, sinks,
                     seed=window)
            c.run()
            assert c.step.status() == (pa.PA_OK, 0)
            c.check()


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("sigma", [2.0**-9, 30.0])
@pytest.mark.parametrize("q", [2, 90])
def test_small_and_large_values(torch, bits, sigma, q):
    c = Case(torch, bits, [q, 1], [q + 90, 200], 8, 2, 128, 128, 16, 60, 5, sigma=sigma, scale=0.01)
    c.run()
    c.check()


# q, ctx, H, Hk, hk, hv, block, window, sinks; (sequence, position) of what is bad
NAN = [
    ([6, 1], [90, 200], 8, 2, 128, 128, 16, 20, 3, [(0, 66), (0, 87), (1, 1)]),
    ([9, 12], [350, 12], 4, 1, 64, 64, 64, 5, 0, [(0, 338), (1, 3), (0, 349)]),
    ([5], [200], 4, 2, 256, 256, 16, 30, 0, [(0, 167), (0, 198)]),
    ([3], [60], 2, 1, 48, 32, 16, 9, 4, [(0, 49), (0, 59)]),
    ([3], [60], 2, 1, 272, 272, 16, 9, 4, [(0, 49), (0, 59)]),
    ([100, 40], [300, 40], 4, 2, 128, 128, 16, 64, 0, [(0, 150), (0, 250), (0, 299), (1, 39)]),
    ([300], [400], 4, 1, 64, 64, 128, 100, 20, [(0, 30), (0, 120), (0, 333), (0, 380)]),
    ([300, 50], [300, 500], 16, 2, 128, 128, 128, 50, 0, [(0, 200), (0, 31), (1, 451)]),
]


@pytest.mark.parametrize("case", NAN, ids=str)
@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("bad", ["key", "value"])
def test_rows_that_do_not_attend_what_is_no_number(torch, bits, case, bad):
    """NaN and infinities in one key or value reach exactly the rows that attend it."""
    *shape, hit = case
    q, ctx, bs, window, sinks = shape[0], shape[1], shape[6], shape[7], shape[8]

    def poison(c, x):
        if (len(c.real) == 0) != (bad == "key"):
            return
        for n, (b, j) in enumerate(hit):
            blk, off = c.batch.slots(b, j, j + 1)
            x[blk[0], off[0], :, n % 3] = [np.nan, np.inf, -np.inf][n % 3]

    c = Case(torch, bits, *shape, poison=poison)
    c.run()
    assert c.step.status() == (pa.PA_OK, 0)
    got = c.out.cpu().numpy()
    touched = np.zeros(len(got), bool)
    for b, j in hit:
        t0 = int(c.batch.starts[b])
        touched[t0:t0 + q[b]] |= wref.sees(q[b], ctx[b], window, sinks)[:, j]
    assert touched.any() and not touched.all()
    assert np.isfinite(got[~touched]).all()
    if bad == "value":
        assert (~np.isfinite(got[touched]).all(axis=(1, 2))).all()
    clean = Case(torch, bits, *shape)
    want, bound = clean.want()
    err = np.abs(got.astype(np.float64) - want)
    assert (err[~touched] <= bound[~touched]).all()


def test_infinite_values_come_through_as_they_are(torch):
    """A row that attends one infinity has it in its output, with its sign; beside another sign NaN."""
    def poison(c, x):
        if len(c.real):
            for j, v in ((70, np.inf), (73, -np.inf)):
                blk, off = c.batch.slots(0, j, j + 1)
                x[blk[0], off[0], :, 2] = v

    for H, q in ((4, 10), (16, 30)):
        ctx, window = 70 + q, 6
        c = Case(torch, 16, [q], [ctx], H, 1, 128, 128, 16, window, 0, poison=poison)
        got = c.run().cpu().numpy()
        see = wref.sees(q, ctx, window, 0)
        for i in range(q):
            a, b = see[i, 70], see[i, 73]
            col = got[i, :, 2]
            assert (np.isnan(col) if a and b else col == np.inf if a else col == -np.inf if b
                    else np.isfinite(col)).all(), i
        assert np.isfinite(np.delete(got, 2, axis=2)).all()


@pytest.mark.parametrize("q", [4, 60])
def test_bad_lengths_and_blocks(torch, q):
    def fresh():
        return Case(torch, 8, [q, 3], [q + 36, 30], 8, 2, 128, 128, 16, 20, 3)
    c = fresh()
    ctx = c.batch.ctx.copy()
    ctx[0] = q - 1
    c.args[2] = up(torch, ctx)
    c.run()
    assert c.step.status() == (pa.PA_ERR_INVALID_ARG, pa.PA_STATUS_BIT_PLAN)
    assert (c.out[:q] == 7).all()
    c.check([1])
    c = fresh()
    tables = c.args[1].clone()
    tables[0, (q + 35) // 16] = c.batch.num_blocks
    c.args[1] = tables
    c.run()
    assert c.step.status() == (pa.PA_ERR_BLOCK_INDEX, pa.PA_STATUS_BIT_BLOCK_INDEX)
    c.check([1])
    # a length that no token belongs to, and fewer rows than the lengths say
    c = fresh()
    c.args[3] = up(torch, np.array([q, -1], np.int32))
    c.run()
    assert c.step.status() == (pa.PA_ERR_INVALID_ARG, pa.PA_STATUS_BIT_PLAN)
    c.check([0])
    c = fresh()
    out = torch.full((q + 1, 8, 128), 7.0, dtype=torch.float16, device="cuda")
    full = c.run().clone()
    assert c.step.status() == (pa.PA_OK, 0)
    c.step.run(c.args[0][:q + 1].contiguous(), *c.args[1:], out)
    assert c.step.status() == (pa.PA_ERR_INVALID_ARG, pa.PA_STATUS_BIT_PLAN)
    assert torch.equal(out, full[:q + 1])


def test_one_token_without_q_seqlens_and_a_larger_bound(torch):
    c = Case(torch, 16, [1, 1, 1], [5, 90, 400], 8, 2, 128, 128, 16, 50, 4)
    want = c.run().clone()
    c.args[3] = None
    assert torch.equal(c.run(), want)
    c.check()
    # the bound on the drafts may be far above what they are (another kernel)
    for max_q in (8, 40, 4000):
        d = Case(torch, 16, [1, 3, 0], [5, 90, 400], 8, 2, 128, 128, 16, 50, 4, max_q=max_q)
        d.run()
        d.check()


@pytest.mark.parametrize("q", [8, 100])
def test_captured_and_replayed_with_other_lengths(torch, q):
    c = Case(torch, 8, [q, q], [900, 900], 8, 2, 128, 128, 64, 10**6, 0)
    s = torch.cuda.Stream()
    c.run(stream=s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        c.run()
    g.replay()
    torch.cuda.synchronize()
    c.check()
    c.batch.ctx[:] = [333, q]  # shorter contexts: the same blocks
    c.args[2].copy_(up(torch, c.batch.ctx))
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    c.check()


def test_two_streams_at_once(torch):
    """Two steps with a workspace each, side by side, give what they give alone."""
    cases = [Case(torch, bits, [q] * 6, [q + 500] * 6, 8, 2, 128, 128, 16, 200, 4, seed=q)
             for bits, q in ((8, 3), (16, 70))]
    alone = [c.run().clone() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(25):
        for c, s in zip(cases, streams):
            c.run(stream=s)
    torch.cuda.synchronize()
    for c, want in zip(cases, alone):
        assert torch.equal(c.out, want)
        c.check()


@pytest.mark.parametrize("bits,H,q,lo,hi,d,window,sinks", [
    (8, 8, 1, 1, 900, 128, 300, 4), (16, 8, 1, 1, 900, 128, 300, 70), (8, 8, 4, 50, 300, 64, 100, 0),
    (16, 8, 2, 50, 300, 256, 100, 40), (8, 12, 5, 50, 300, 96, 64, 3), (8, 32, 8, 100, 700, 128, 129, 4),
    (16, 32, 64, 0, 700, 128, 200, 4), (8, 32, 64, 0, 700, 128, 200, 4), (16, 4, 200, 0, 300, 64, 150, 33),
    (8, 4, 200, 0, 300, 64, 150, 0)])
def test_again_and_again(torch, bits, H, q, lo, hi, d, window, sinks):
    """Many row tiles whose ends leave no pause in the rings: a hundred runs give the same bits, and
    every twentieth sequence is attention in 64 bits."""
    rng = np.random.default_rng(q + H)
    qs = rng.integers(max(1, q // 2), q + 1, 120)
    c = Case(torch, bits, qs, qs + rng.integers(lo, hi, 120), H, 2, d, d, 16, window, sinks)
    first = c.run().clone().view(torch.int16)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(100):
        differ += (c.run().view(torch.int16) != first).any()
    assert differ.item() == 0
    assert c.step.status() == (pa.PA_OK, 0)
    c.check(list(range(0, 120, 20)))


@pytest.mark.parametrize("shape", [(8, 2, 64, 2), (16, 1, 128, 8), (16, 1, 64, 20), (4, 2, 272, 3)], ids=str)
def test_slots_that_were_never_written_are_zero_rows(torch, shape):
    """Zero codes under zero exponent bytes amid a window."""
    H, Hk, d, q = shape
    c = Case(torch, 8, [q, q, 1], [400, 290, 9], H, Hk, d, d, 16, 150, 20)
    for n, (codes, exps) in enumerate(c.dev):
        for b, lo, hi in ((0, 3, 9), (0, 300, 390), (1, 250, 251), (2, 0, 9)):
            blk, off = c.batch.slots(b, lo, hi)
            codes.view(torch.uint8)[blk, off] = 0
            exps.transpose(1, 2)[blk, off] = 0
            c.real[n][blk, off] = 0
            c.exp[n].transpose(0, 2, 1)[blk, off] = -127
    c.run()
    assert c.step.status() == (pa.PA_OK, 0)
    c.check()


@pytest.mark.parametrize("case", [([3, 2], [290, 40], 8, 2, 128, 16), ([20, 7, 1], [150, 263, 128], 8, 4, 64, 48),
                                  ([200], [500], 4, 1, 128, 64)], ids=str)
@pytest.mark.parametrize("spread", [(0, 8), (0, 15), (-24, 16)], ids=str)
def test_rows_of_many_magnitudes(torch, case, spread):
    q, ctx, H, Hk, d, bs = case
    c = Case(torch, 8, q, ctx, H, Hk, d, d, bs, 70, 20, spread=spread, scale=2.0 ** -(spread[1] + 9))
    c.run()
    assert c.step.status() == (pa.PA_OK, 0)
    c.check()


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("q", [3, 50])
def test_large_rows_outside_the_window_take_nothing_from_those_in_it(torch, bits, q):
    """A key and a value of fp16's largest size just outside the windows of most rows."""
    def poison(c, x):
        if len(c.real):
            x *= np.float16(2.0**-9)
        blk, off = c.batch.slots(0, 200, 201)
        x[blk[0], off[0]] = np.where(x[blk[0], off[0]] < 0, -65504, 65504)

    window = 220 + q // 2 - 200
    c = Case(torch, bits, [q], [220 + q], 8, 1, 128, 128, 16, window, 0, poison=poison)
    c.run()
    want, bound = c.want()
    err = np.abs(c.out.cpu().numpy().astype(np.float64) - want)
    far = ~wref.sees(q, 220 + q, window, 0)[:, 200]
    assert far.any() and not far.all()
    assert (err[far] <= bound[far]).all()


def test_long_cache_past_32_bit_offsets(torch):
    """Blocks whose bytes lie behind 2^32 and whose elements lie behind 2^31."""
    bs, Hk, d = 128, 32, 128
    nb = (2**32 + 2**31) // (bs * Hk * d * 2) + 40
    k, v = (torch.zeros((nb, bs, Hk, d), dtype=torch.float16, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(3)
    for q in (1, 70):
        blocks = np.array([[nb - 1, 5, nb - 7, nb - 2, 9]], np.int32)
        for b in blocks[0]:
            k[b] = torch.randn((bs, Hk, d), generator=g, device="cuda").half()
            v[b] = torch.randn((bs, Hk, d), generator=g, device="cuda").half()
        batch = ref.Batch(np.arange(5, dtype=np.int32)[None], np.array([600], np.int32), np.array([q], np.int32), bs, 5)
        x = torch.randn((q, Hk, d), generator=g, device="cuda").half()
        step = pa.WindowStep(k, v, batch=1, num_heads=Hk, max_seqlen_q=q, max_blocks_per_seq=5, window=300, sinks=3)
        out = torch.empty_like(x)
        step.run(x, up(torch, blocks), up(torch, batch.ctx), up(torch, batch.q), out)
        assert step.status() == (pa.PA_OK, 0)
        rows = torch.from_numpy(blocks[0].astype(np.int64)).cuda()
        want, bound = wref.window_attention(x.cpu().numpy(), k[rows].double().cpu().numpy(),
                                            v[rows].double().cpu().numpy(), np.zeros((5, Hk, bs)), batch, 300, 3,
                                            1 / math.sqrt(d))
        assert (np.abs(out.cpu().numpy() - want) <= bound).all()


def test_a_window_model_serves(torch):
    """Prompts in parts, decode steps and drafts of several requests over one 8-bit cache whose blocks
    the pool hands out and takes back: every step's outputs are attention in 64 bits over the rows
    that the cache was given, and no more blocks are held than the windows need."""
    rng = np.random.default_rng(0)
    H, Hk, d, bs, window, sinks, rows = 8, 2, 128, 16, 50, 20, 4
    sections = (16, 24, 24)
    nb, cols = 60, 40
    pool = pa.BlockPool.empty(rows, cols, nb, bs, window=window, sinks=sinks)
    cache = pa.QuantCache.empty(nb, bs, Hk, d)
    angle = np.arange(800)[:, None] * 10000.0 ** (-np.arange(0, d, 2) / d)
    cs = np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)
    w = (1 + 0.1 * rng.normal(size=d)).astype(np.float16)
    ctx = np.zeros(rows, np.int32)
    hist = [[] for _ in range(rows)]  # of a request: dequantised (key, value, value exponent) rows
    for n in range(14):
        q = np.zeros(rows, np.int32)
        for b in range(rows):
            if ctx[b] > 300 and n % 4 == 3:
                ctx[b], hist[b] = 0, []
            else:
                q[b] = rng.choice([1, 3, 60, 100]) if n else rng.integers(1, 100)
        ctx = ctx + q
        T = int(q.sum())
        lens, qs, pad = up(torch, ctx), up(torch, q), 3
        slots = torch.empty(T + pad, dtype=torch.int64, device="cuda")
        pos = torch.empty(T + pad, dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        pool.step(lens, qs, slots, pos, status=status)
        # text: all axes alike; the second request has images: the height moves on its own
        places = pos.repeat(3, 1)
        t1 = int(q[:1].sum())
        places[1, t1:t1 + int(q[1])] = (places[1, t1:t1 + int(q[1])] * 7) % 31
        x = rng.normal(size=(T + pad, H + 2 * Hk, d)).astype(np.float16)
        dx = up(torch, x)
        qo = torch.zeros((T + pad, H, d), dtype=torch.float16, device="cuda")
        cache.store(dx[:, :H], dx[:, H:H + Hk], dx[:, H + Hk:], up(torch, w), up(torch, w), up(torch, cs), places,
                    pool.block_tables, lens, qs, int(max(q.max(), 1)), qo, status=status, sections=sections)
        step = pa.WindowStep(cache.key, cache.value, cache.key_exps, cache.value_exps, batch=rows, num_heads=H,
                             max_seqlen_q=int(max(q.max(), 1)), max_blocks_per_seq=cols, window=window, sinks=sinks)
        out = torch.full((T + pad, H, d), 7.0, dtype=torch.float16, device="cuda")
        step.run(qo, pool.block_tables, lens, qs, out)
        assert step.status() == (pa.PA_OK, 0) and status.item() == 0
        assert bool((out[T:] == 7).all()) and bool((qo[T:] == 0).all()) and pos[T:].tolist() == [-1] * pad
        # the rows that went into the cache, read at the slots that the pool named
        at = slots[:T].cpu().numpy()
        assert (at >= 0).all()
        key, val = (ref.decode(t.view(torch.uint8).cpu().numpy()) for t in (cache.key, cache.value))
        ke, ve = (t.cpu().numpy().astype(np.int64) - 127 for t in (cache.key_exps, cache.value_exps))
        t = 0
        for b in range(rows):
            for _ in range(q[b]):
                blk, off = at[t] // bs, at[t] % bs
                hist[b].append((key[blk, off] * 2.0 ** ke[blk, :, off][:, None],
                                val[blk, off] * 2.0 ** ve[blk, :, off][:, None], ve[blk, :, off]))
                t += 1
            assert len(hist[b]) == ctx[b]
        # keys: what was projected, turned by its positions and quantised (2^-4 of the value)
        turned, _ = wref.rotate_axes(x[:T, H:H + Hk], w, cs, places[:, :T].cpu().numpy(), sections, False, 1e-6, False)
        new = np.concatenate([np.stack([r[0] for r in hist[b][ctx[b] - q[b]:]]) for b in range(rows) if q[b]])
        top = np.abs(turned).max(-1, keepdims=True)
        assert (np.abs(new - turned) <= 1.001 * 2.0**-4 * np.abs(turned) + 2.0**-17 * top).all()
        # attention over the requests' own rows, as caches of one block each
        most = int(max(ctx.max(), 1))
        most += -most % 16
        k64, v64, e64 = np.zeros((rows, most, Hk, d)), np.zeros((rows, most, Hk, d)), np.zeros((rows, Hk, most))
        for b in range(rows):
            for i, (kk, vv, ee) in enumerate(hist[b]):
                k64[b, i], v64[b, i], e64[b, :, i] = kk, vv, ee
        flat = ref.Batch(np.arange(rows, dtype=np.int32)[:, None], ctx, q, most, rows)
        want, bound = wref.window_attention(qo[:T].cpu().numpy(), k64, v64, e64, flat, window, sinks, 1 / math.sqrt(d))
        assert (np.abs(out[:T].cpu().numpy() - want) <= bound).all()
        held, gone = pool.held.cpu().numpy(), pool.gone.cpu().numpy()
        assert (held - gone <= -(-sinks // bs) + -(-(window + q) // bs) + 1).all()
        assert pool.count.item() == nb - int((held - gone).sum())
