"""pa_blocks_step at the ends of what it takes: numbers of blocks that leave some lanes a last round of their own,
as many rows as there may be, tables near 2^31 entries."""
import numpy as np
import pytest

import paged_kv_cache_206_gb300 as pa
from . import window_ref as wref
from .test_gpu_blocks import same, step
from .test_gpu_cache import up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    torch.cuda.set_device(0)
    return torch


@pytest.mark.parametrize("back", [1, 31, 33, 511, 4095, 4097, 4096 + 511, 3 * 4096 + 17])
def test_blocks_given_back_that_fill_no_round(torch, back):
    """So many blocks of nine rows come back while a tenth row's are handed out, then with every third
    entry naming no block."""
    held = np.append(np.random.default_rng(back).multinomial(back, [1 / 9] * 9), 0)
    cols, blocks = int(held.max()) + 1, back + int(held.max()) + 1
    pool, want = pa.BlockPool.empty(10, cols, blocks, 16), wref.Pool(10, cols, blocks, 16)
    ctx, end = (16 * held).tolist(), [0] * 9 + [16 * cols]
    for _ in range(3):
        assert not step(torch, pool, want, ctx, ctx)
        assert not step(torch, pool, want, end, end)
    assert not step(torch, pool, want, ctx, ctx)
    spoiled = pool.block_tables.clone()
    lost = 0
    for b in range(9):
        spoiled[b, :held[b]:3] = blocks + b
        lost += -(-int(held[b]) // 3)
    pool.block_tables.copy_(spoiled)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool.step(torch.zeros(10, dtype=torch.int32, device="cuda"), status=status)
    assert status.item() == pa.PA_STATUS_BIT_BLOCK_INDEX
    assert pool.count.item() == blocks and bool((pool.block_tables == -1).all())
    free = pool.free.tolist()
    assert free.count(-1) == lost and len(set(free) - {-1}) == blocks - lost


def test_as_many_entries_given_back_as_a_table_may_have(torch):
    """Rows that say that they hold every entry of a table of 2^31 - 2048, none of which names a block."""
    rows, cols, blocks = 2048, 2**20 - 1, 16
    tables = torch.full((rows, cols), -5, dtype=torch.int32, device="cuda")
    held = torch.full((rows,), cols, dtype=torch.int32, device="cuda")
    gone = torch.zeros_like(held)
    free = torch.full((blocks,), 7, dtype=torch.int32, device="cuda")
    count = torch.zeros(1, dtype=torch.int32, device="cuda")
    pool = pa.BlockPool(tables, held, gone, free, count, block_size=16)
    pool.step(torch.zeros_like(held))
    assert all(bool((part == -1).all()) for part in tables.split(64))
    assert bool((held == 0).all()) and count.item() == blocks and free.tolist() == [-1] * blocks


@pytest.mark.parametrize("rows", [1025, 1537, 1756, 2048])
@pytest.mark.parametrize("window", [0, 40])
def test_as_many_rows_as_there_may_be(torch, rows, window):
    """Three and four rows a thread, and (from 1756 rows on) more than 48 KB of shared memory: with slots of
    few tokens and of many, and without. Some rows begin anew without a step of length 0 between, so that with a
    window current tokens lie where blocks were given back: they have no slot, and the status says so."""
    rng = np.random.default_rng(rows)
    bs, cols = 16, 12
    pool, want = pa.BlockPool.empty(rows, cols, rows * 5, bs, window=window, sinks=3), \
        wref.Pool(rows, cols, rows * 5, bs, window, 3)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def go(ctx, q, tokens, outs):
        slots = torch.full((tokens,), 77, dtype=torch.int64, device="cuda") if outs else None
        pos = torch.full((tokens,), 77, dtype=torch.int32, device="cuda") if outs else None
        status.zero_()
        pool.step(up(torch, ctx.astype(np.int32)), None if q is None else up(torch, q.astype(np.int32)), slots, pos,
                  status=status)
        want_slots, want_pos, out_of = want.step(ctx.tolist(), None if q is None else q.tolist(), tokens)
        same(pool, want)
        bits = pa.PA_STATUS_BIT_POOL if out_of else 0
        if outs:
            assert slots.tolist() == want_slots and pos.tolist() == want_pos
            for b, n in enumerate(np.minimum(ctx, 1) if q is None else q):
                pages = range(int(ctx[b] - n) // bs, min(-(-int(ctx[b]) // bs), want.held[b]))
                if n and any(want.tables[b][page] < 0 for page in pages):
                    bits |= pa.PA_STATUS_BIT_BLOCK_INDEX
        assert status.item() == bits
        return bits

    ctx, seen = np.zeros(rows, int), 0
    for n in range(8):
        q = np.where(rng.random(rows) < 0.7, rng.choice([1, 1, 5, 40], rows), 0)
        ctx = np.where(rng.random(rows) < 0.15, 0, ctx)
        q = np.where(ctx + q > cols * bs, 0, q)
        ctx = ctx + q
        seen |= go(ctx, q, int(q.sum()) + n % 3, n % 4 != 3)
    assert (seen & pa.PA_STATUS_BIT_BLOCK_INDEX != 0) == (window > 0)
    one = np.minimum(ctx + 1, cols * bs)
    go(np.where(rng.random(rows) < 0.2, 0, one), None, rows, True)  # one token a row
    go(np.zeros(rows, int), np.zeros(rows, int), 0, False)
    assert sorted(pool.free.tolist()) == list(range(rows * 5))


@pytest.mark.parametrize("rows", [1300, 2048])
def test_as_many_rows_captured(torch, rows):
    bs, cols = 16, 8
    pool, want = pa.BlockPool.empty(rows, cols, rows * cols, bs), wref.Pool(rows, cols, rows * cols, bs)
    lens, q = (torch.zeros(rows, dtype=torch.int32, device="cuda") for _ in range(2))
    slots = torch.empty(3 * rows, dtype=torch.int64, device="cuda")
    pos = torch.empty(3 * rows, dtype=torch.int32, device="cuda")
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    pool.step(lens, q, slots, pos, stream=s)
    s.synchronize()
    with torch.cuda.graph(g, stream=s):
        pool.step(lens, q, slots, pos)
    rng, ctx = np.random.default_rng(rows), np.zeros(rows, int)
    for _ in range(6):
        n = rng.integers(0, 4, rows)
        ctx += n
        lens.copy_(up(torch, ctx.astype(np.int32)))
        q.copy_(up(torch, n.astype(np.int32)))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want_slots, want_pos, _ = want.step(ctx.tolist(), n.tolist(), 3 * rows)
        same(pool, want)
        assert slots.tolist() == want_slots and pos.tolist() == want_pos
