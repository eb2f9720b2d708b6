"""pa_blocks_step against the pool told in lists: many steps of requests that come, grow, move
on with their window and end."""
import numpy as np
import pytest

import paged_kv_cache_206_gb300 as pa
from . import window_ref as wref
from .test_gpu_cache import up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    torch.cuda.set_device(0)
    return torch


def same(pool, want):
    np.testing.assert_array_equal(pool.block_tables.cpu().numpy(), np.array(want.tables))
    np.testing.assert_array_equal(pool.held.cpu().numpy(), want.held)
    np.testing.assert_array_equal(pool.gone.cpu().numpy(), want.gone)
    assert pool.count.item() == want.count
    np.testing.assert_array_equal(pool.free.cpu().numpy(), want.free)


def step(torch, pool, want, ctx, q, extra=0, stream=None, outs=True):
    """One step of both; whether blocks ran out."""
    tokens = (sum(q) if q is not None else len(ctx)) + extra
    slots = torch.full((tokens,), 77, dtype=torch.int64, device="cuda") if outs else None
    pos = torch.full((tokens,), 77, dtype=torch.int32, device="cuda") if outs else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = up(torch, np.array(ctx, np.int32))
    qs = None if q is None else up(torch, np.array(q, np.int32))
    torch.cuda.synchronize()
    pool.step(lens, qs, slots, pos, status=status, stream=stream)
    torch.cuda.synchronize()
    want_slots, want_pos, out_of = want.step(list(ctx), None if q is None else list(q), tokens)
    same(pool, want)
    if outs:
        assert slots.tolist() == want_slots and pos.tolist() == want_pos
    assert status.item() == (pa.PA_STATUS_BIT_POOL if out_of else 0)
    return out_of


# rows, blocks, block size, window, sinks, longest prompt
CASES = [(1, 40, 16, 0, 0, 300), (3, 60, 16, 40, 4, 200), (7, 500, 48, 100, 50, 1500), (64, 700, 16, 33, 0, 120),
         (300, 4000, 16, 64, 17, 200), (40, 900, 128, 1, 0, 2000), (513, 3000, 16, 0, 0, 60), (5, 30, 16, 16, 500, 90)]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_requests_come_and_go(torch, case):
    rows, blocks, bs, window, sinks, longest = case
    rng = np.random.default_rng(rows + bs)
    cols = -(-longest // bs) + 3
    pool = pa.BlockPool.empty(rows, cols, blocks, bs, window=window, sinks=sinks)
    want = wref.Pool(rows, cols, blocks, bs, window, sinks)
    ctx, ran_out = np.zeros(rows, int), 0
    for n in range(25):
        q = np.zeros(rows, int)
        for b in range(rows):
            kind = rng.random()
            if ctx[b] == 0:
                if kind < 0.5:  # a prompt
                    ctx[b] = q[b] = rng.integers(1, longest + 1)
            elif kind < 0.2:
                ctx[b] = 0
            elif kind < 0.9:  # a token, drafts, or a part of a prompt
                q[b] = rng.choice([1, 1, rng.integers(1, 20), rng.integers(1, longest)])
                if ctx[b] + q[b] > cols * bs:
                    q[b] = 0
                ctx[b] += q[b]
        ran_out += step(torch, pool, want, ctx, q, extra=int(rng.integers(0, 4)), outs=n % 5 != 4)
    step(torch, pool, want, np.zeros(rows, int), np.zeros(rows, int))
    assert pool.count.item() == blocks
    assert sorted(pool.free.tolist()) == list(range(blocks))


def test_an_empty_pool_says_so_and_goes_on_later(torch):
    pool, want = pa.BlockPool.empty(4, 8, 9, 16), wref.Pool(4, 8, 9, 16)
    assert step(torch, pool, want, [50, 70, 20, 1], [50, 70, 20, 1])
    assert pool.held.tolist() == [4, 5, 0, 0] and pool.count.item() == 0
    assert step(torch, pool, want, [51, 71, 20, 1], [1, 1, 20, 1])
    assert not step(torch, pool, want, [0, 71, 20, 1], [0, 0, 20, 1])
    assert pool.held.tolist() == [0, 5, 2, 1]


def test_lengths_alone_say_one_token_a_row(torch):
    pool, want = pa.BlockPool.empty(5, 4, 30, 16), wref.Pool(5, 4, 30, 16)
    for ctx in ([1, 0, 16, 17, 64], [2, 1, 17, 0, 64], [0, 0, 0, 0, 0]):
        step(torch, pool, want, ctx, None, extra=2)


def test_what_was_taken_in_one_step_and_given_back_leaves_the_stack(torch):
    pool = pa.BlockPool.empty(30, 40, 1200, 16)
    pool.free.copy_(torch.randperm(1200, device="cuda").to(torch.int32))
    before = pool.free.clone()
    lens = torch.randint(1, 600, (30,), device="cuda").to(torch.int32)
    for _ in range(3):
        pool.step(lens, lens)
        assert pool.count.item() == 1200 - int(((lens + 15) // 16).sum())
        pool.step(torch.zeros_like(lens), torch.zeros_like(lens))
        assert torch.equal(pool.free, before) and pool.count.item() == 1200


def test_lengths_and_states_that_break_a_constraint(torch):
    """Their rows stay as they are, their tokens get -1, and the others are what they are without them."""
    good = wref.Pool(6, 4, 30, 16)
    pool = pa.BlockPool.empty(6, 4, 30, 16)
    step(torch, pool, good, [10, 20, 30, 40, 50, 60], [10, 20, 30, 40, 50, 60])
    pool.gone[5] = 3  # (with 4 entries held: three of them gone)
    pool.held[4] = 5
    ctx, q = [11, 19, 31, 65, 51, 61], [1, 20, -1, 25, 1, 1]
    slots = torch.full((60,), 7, dtype=torch.int64, device="cuda")
    pos = torch.full((60,), 7, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tables = pool.block_tables.clone()
    pool.step(up(torch, np.array(ctx, np.int32)), up(torch, np.array(q, np.int32)), slots, pos, status=status)
    # row 5's state is in order (no sinks): its entry 3 is still held
    assert status.item() == pa.PA_STATUS_BIT_PLAN and pa.pa_status_read(status)[0] == pa.PA_ERR_INVALID_ARG
    assert torch.equal(pool.block_tables, tables) and pool.held.tolist() == [1, 2, 2, 3, 5, 4]
    want = [-1] * 60
    want[0], want[47] = tables[0, 0].item() * 16 + 10, tables[5, 3].item() * 16 + 12
    assert slots.tolist() == want
    assert [i for i, p in enumerate(pos.tolist()) if p != -1] == [0, 47]


def test_more_tokens_than_there_are_rows_for(torch):
    pool, status = pa.BlockPool.empty(3, 4, 30, 16), torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = up(torch, np.array([5, 2**31 - 1, 7], np.int32))
    slots = torch.full((6,), 7, dtype=torch.int64, device="cuda")
    pool.step(lens, lens, slots, status=status)
    assert status.item() == pa.PA_STATUS_BIT_PLAN
    assert slots.tolist() == [0, 1, 2, 3, 4, -1] and pool.held.tolist() == [1, 0, 1]
    # no slots are asked for: nothing to run over
    status.zero_()
    lens = up(torch, np.array([5, 6, 7], np.int32))
    pool.step(lens, lens, status=status)
    assert status.item() == 0 and pool.held.tolist() == [1, 1, 1]


def test_bad_entries_and_counts(torch):
    pool, status = pa.BlockPool.empty(2, 4, 8, 16), torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = up(torch, np.array([40, 20], np.int32))
    pool.step(lens, lens, status=status)
    assert status.item() == 0
    pool.block_tables[0, 1] = 8
    slots = torch.empty(2, dtype=torch.int64, device="cuda")
    pool.step(up(torch, np.array([18, 21], np.int32)), up(torch, np.ones(2, np.int32)), slots, status=status)
    assert status.item() == pa.PA_STATUS_BIT_BLOCK_INDEX
    assert slots[0].item() == -1 and slots[1].item() >= 0
    status.zero_()
    pool.step(torch.zeros_like(lens), torch.zeros_like(lens), status=status)
    assert status.item() == pa.PA_STATUS_BIT_BLOCK_INDEX and pool.count.item() == 8
    assert sorted(pool.free.tolist()) == [-1, 0, 2, 3, 4, 5, 6, 7]
    for count in (-5, 9, 2**31 - 1):
        status.zero_()
        pool.count.fill_(count)
        pool.step(torch.zeros_like(lens), torch.zeros_like(lens), status=status)
        assert status.item() == pa.PA_STATUS_BIT_POOL
        assert pool.count.item() == (0 if count < 0 else 8)


@pytest.mark.parametrize("rows,tokens", [(4, 12), (700, 2500)])
def test_captured_and_replayed(torch, rows, tokens):
    """A captured step follows the lengths that it is replayed with, on its own stream."""
    pool, want = pa.BlockPool.empty(rows, 20, rows * 12, 16, window=20, sinks=2), \
        wref.Pool(rows, 20, rows * 12, 16, 20, 2)
    lens, q = (torch.zeros(rows, dtype=torch.int32, device="cuda") for _ in range(2))
    slots = torch.empty(tokens, dtype=torch.int64, device="cuda")
    pos = torch.empty(tokens, dtype=torch.int32, device="cuda")
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    pool.step(lens, q, slots, pos, stream=s)
    s.synchronize()
    with torch.cuda.graph(g, stream=s):
        pool.step(lens, q, slots, pos)
    rng, ctx = np.random.default_rng(rows), np.zeros(rows, int)
    for _ in range(12):
        n = rng.integers(0, 4, rows)
        ctx += n
        lens.copy_(up(torch, ctx.astype(np.int32)))
        q.copy_(up(torch, n.astype(np.int32)))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want_slots, want_pos, _ = want.step(ctx.tolist(), n.tolist(), tokens)
        same(pool, want)
        assert slots.tolist() == want_slots and pos.tolist() == want_pos


def test_two_pools_on_two_streams(torch):
    pools = [pa.BlockPool.empty(50, 70, 3000, 16) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in pools]
    lens = torch.randint(1, 900, (50,), device="cuda").to(torch.int32)
    slots = [torch.empty(int(lens.sum()), dtype=torch.int64, device="cuda") for _ in pools]
    torch.cuda.synchronize()
    for _ in range(10):
        for p, s, out in zip(pools, streams, slots):
            p.step(lens, lens, out, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(slots[0], slots[1]) and torch.equal(pools[0].block_tables, pools[1].block_tables)
    assert len(set(slots[0].tolist())) == slots[0].numel()
