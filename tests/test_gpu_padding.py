"""Rows without a context where no lengths of current tokens are given: padding, to the pool, to the cache
and to the attention alike, so that a captured decode loop goes on as requests end."""
import numpy as np
import pytest

import paged_kv_cache_206_gb300 as pa
from . import serving_ref as ref
from .test_gpu_cache import empty_cache, expected_cache, rows
from .test_gpu_window import Case, up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    torch.cuda.set_device(0)
    return torch


# contexts; one that begins with padding, one of more than 32 and one of more than 128 rows
BATCHES = [[5, 0, 90, 0, 400], [0, 0, 33], [0] + [7, 0, 60, 129] * 9, [40, 0, 1] * 50 + [0]]


@pytest.mark.parametrize("ctx", BATCHES, ids=len)
@pytest.mark.parametrize("shape", [(8, 2, 128), (8, 2, 64), (16, 1, 256), (40, 1, 128), (64, 1, 64), (200, 1, 128),
                                   (4, 2, 272)], ids=str)
@pytest.mark.parametrize("bits", [8, 16])
def test_the_attention_leaves_them_out(torch, bits, shape, ctx):
    H, Hk, d = shape
    live = np.array(ctx) > 0
    c = Case(torch, bits, live.astype(int), ctx, H, Hk, d, d, 16, 50, 4, max_q=1)
    want = c.run().clone()
    assert c.step.status() == (pa.PA_OK, 0)
    c.check()
    query = torch.zeros((len(ctx), H, d), dtype=torch.float16, device="cuda")
    query[up(torch, live)] = c.args[0][:c.tokens]
    out = torch.full_like(query, 7.0)
    c.step.run(query, *c.args[1:3], None, out)
    assert c.step.status() == (pa.PA_OK, 0)
    assert torch.equal(out[up(torch, live)], want[:c.tokens])
    assert bool((out[up(torch, ~live)] == 7).all())


@pytest.mark.parametrize("ctx", BATCHES, ids=len)
@pytest.mark.parametrize("shape", [(8, 2, 128), (40, 1, 128), (200, 1, 64), (4, 2, 272)], ids=str)
@pytest.mark.parametrize("bits", [8, 16])
def test_so_does_the_attention_of_drafts(torch, bits, shape, ctx):
    H, Hk, d = shape
    live = np.array(ctx) > 0
    c = Case(torch, bits, live.astype(int), ctx, H, Hk, d, d, 16, 2**31 - 1, 0, max_q=1)
    (k, ke), (v, ve) = c.dev
    step = pa.TreeStep(k, v, ke, ve, batch=len(ctx), num_heads=H, max_seqlen_q=1,
                       max_blocks_per_seq=c.batch.tables.shape[1])
    want = torch.full_like(c.args[0][:c.tokens], 7.0)
    step.run(c.args[0][:c.tokens], *c.args[1:4], None, want)
    assert step.status() == (pa.PA_OK, 0)
    query = torch.zeros((len(ctx), H, d), dtype=torch.float16, device="cuda")
    query[up(torch, live)] = c.args[0][:c.tokens]
    out = torch.full_like(query, 7.0)
    step.run(query, *c.args[1:3], None, None, out)
    assert step.status() == (pa.PA_OK, 0)
    assert torch.equal(out[up(torch, live)], want)
    assert bool((out[up(torch, ~live)] == 7).all())


@pytest.mark.parametrize("ctx", BATCHES, ids=len)
@pytest.mark.parametrize("call", ["write", "store", "axes"])
def test_the_cache_leaves_them_out(torch, call, ctx):
    H, Hk, d, bs = 4, 2, 64, 16
    rng = np.random.default_rng(len(ctx))
    live = np.array(ctx) > 0
    batch = ref.make_batch(rng, live.astype(int), ctx, bs)
    n = len(ctx)
    xq, k, v = rows(rng, n, H, d), rows(rng, n, Hk, d), rows(rng, n, Hk, d)
    c = empty_cache(torch, batch.num_blocks, bs, Hk, d, d)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = up(torch, batch.tables), up(torch, batch.ctx), None, 1
    qo = torch.full((n, H, d), 7.0, dtype=torch.float16, device="cuda")
    if call == "write":
        c.write(up(torch, k), up(torch, v), *lens, status=status)
    else:  # no norm, no rotation: the rows themselves
        more = {}
        if call == "axes":
            more = dict(sections=(0, 0))
        pos = torch.zeros((2, n), dtype=torch.int32, device="cuda") if more else None
        c.store(up(torch, xq), up(torch, k), up(torch, v), None, None, None, pos, *lens, qo, status=status, **more)
        got = qo.cpu().numpy()
        np.testing.assert_array_equal(got[live], xq[live])
        assert (got[~live] == 7).all()
    assert status.item() == 0
    for x, codes, exps in ((k, c.key, c.key_exps), (v, c.value, c.value_exps)):
        want, want_e = expected_cache(batch, x[live], d, Hk)
        assert ref.same_codes(codes.view(torch.uint8).cpu().numpy(), want)
        np.testing.assert_array_equal(exps.cpu().numpy(), want_e)


@pytest.mark.parametrize("window", [0, 40])
def test_a_captured_decode_loop_goes_on_as_requests_end(torch, window):
    """Pool, store and attention of one token a row, captured once; rows end and begin between the replays. No
    step reports anything, and each one's outputs are those of the same rows alone."""
    rng = np.random.default_rng(window)
    H, Hk, d, bs, n, cols = 8, 2, 64, 16, 6, 12
    pool = pa.BlockPool.empty(n, cols, n * cols, bs, window=window, sinks=3)
    cache = pa.QuantCache.empty(n * cols, bs, Hk, d)
    win = pa.WindowStep(cache.key, cache.value, cache.key_exps, cache.value_exps, batch=n, num_heads=H,
                        max_seqlen_q=1, max_blocks_per_seq=cols, window=window or 2**31 - 1, sinks=3)
    x = torch.zeros((n, H + 2 * Hk, d), dtype=torch.float16, device="cuda")
    lens = torch.zeros(n, dtype=torch.int32, device="cuda")
    slots = torch.zeros(n, dtype=torch.int64, device="cuda")
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qo = torch.full((n, H, d), 7.0, dtype=torch.float16, device="cuda")
    out = torch.full_like(qo, 7.0)

    def step():
        pool.step(lens, None, slots, pos, status=status)
        cache.store(x[:, :H], x[:, H:H + Hk], x[:, H + Hk:], None, None, None, None, pool.block_tables, lens, None, 1,
                    qo, status=status)
        win.run(qo, pool.block_tables, lens, None, out)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()  # nothing runs yet: all padding
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
    ctx = np.zeros(n, np.int32)
    for k in range(60):
        for b in range(n):
            if ctx[b] and rng.random() < 0.03:
                ctx[b] = 0
            elif ctx[b] or rng.random() < 0.3:
                ctx[b] += 1
        live = ctx > 0
        lens.copy_(up(torch, ctx))
        x.copy_(torch.from_numpy(rng.normal(size=x.shape).astype(np.float16)))
        out.fill_(7)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert status.item() == 0 and win.status() == (pa.PA_OK, 0)
        assert pos.tolist() == [c - 1 for c in ctx.tolist()]
        assert ((slots.cpu().numpy() >= 0) == live).all()
        assert bool((out[up(torch, ~live)] == 7).all())
        if live.any():
            alone = torch.full((int(live.sum()), H, d), 7.0, dtype=torch.float16, device="cuda")
            one = pa.WindowStep(cache.key, cache.value, cache.key_exps, cache.value_exps, batch=n, num_heads=H,
                                max_seqlen_q=1, max_blocks_per_seq=cols, window=window or 2**31 - 1, sinks=3)
            one.run(qo[up(torch, live)], pool.block_tables, lens, up(torch, live.astype(np.int32)), alone)
            assert one.status() == (pa.PA_OK, 0)
            assert torch.equal(out[up(torch, live)], alone)
    assert ctx.max() > 20 and (ctx == 0).any()
