"""Lengths that break a constraint, in the serving calls: the sequence is left out, its rows
count where the next one's begin, and the others are right."""
import numpy as np
import pytest

import paged_kv_cache_206_gb300 as pa
from . import serving_ref as ref
from .test_gpu_cache import empty_cache, expected_cache, rows, up
from .test_gpu_tree import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    torch.cuda.set_device(0)
    return torch


# stated lengths, the bound; the batches past 32 and 128 sequences are searched in rounds
LONG = [
    ([5, 2], 3),
    ([1, 9, 3, 0, 2], 4),
    ([6] + [2] * 40, 5),
    ([1] * 130 + [7, 3, 1] + [2] * 20, 4),
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: f"{len(c[0])}")
@pytest.mark.parametrize("call", ["write", "store"])
def test_a_sequence_that_is_too_long_moves_no_other_in_the_cache(torch, call, case):
    q, bound = case
    rng = np.random.default_rng(len(q))
    Hk, H, d, bs = 2, 4, 64, 16
    batch = ref.make_batch(rng, q, [n + int(x) for n, x in zip(q, rng.integers(0, 40, len(q)))], bs)
    T = int(batch.q.sum())
    xq, k, v = rows(rng, T, H, d), rows(rng, T, Hk, d), rows(rng, T, Hk, d)
    c = empty_cache(torch, batch.num_blocks, bs, Hk, d, d)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = up(torch, batch.tables), up(torch, batch.ctx), up(torch, batch.q), bound
    qo = torch.full((T, H, d), 7.0, dtype=torch.float16, device="cuda")
    if call == "write":
        c.write(up(torch, k), up(torch, v), *lens, status=status)
    else:  # no norm, no rotation: the rows themselves
        c.store(up(torch, xq), up(torch, k), up(torch, v), None, None, None, None, *lens, qo, status=status)
    assert status.item() == pa.PA_STATUS_BIT_PLAN
    live = np.repeat(batch.q <= bound, batch.q)
    good = ref.Batch(batch.tables, batch.ctx, np.where(batch.q <= bound, batch.q, 0), bs, batch.num_blocks)
    for x, codes, exps in ((k, c.key, c.key_exps), (v, c.value, c.value_exps)):
        want, want_e = expected_cache(good, x[live], d, Hk)
        assert ref.same_codes(codes.view(torch.uint8).cpu().numpy(), want)
        np.testing.assert_array_equal(exps.cpu().numpy(), want_e)
    if call == "store":
        got = qo.cpu().numpy()
        np.testing.assert_array_equal(got[live], xq[live])
        assert (got[~live] == 7).all()


@pytest.mark.parametrize("case", LONG, ids=lambda c: f"{len(c[0])}")
@pytest.mark.parametrize("shape", [(4, 2, 64), (8, 2, 128), (32, 4, 128), (2, 1, 272)], ids=str)
@pytest.mark.parametrize("bits", [8, 16])
def test_a_sequence_that_is_too_long_moves_no_other_in_the_attention(torch, bits, shape, case):
    q, bound = case
    H, Hk, d = shape
    rng = np.random.default_rng(len(q))
    c = Case(torch, bits, q, [n + int(x) for n, x in zip(q, rng.integers(0, 40, len(q)))], H, Hk, d, d, 16,
             "tree", behind=1)
    (k, ke), (v, ve) = c.dev
    c.step = pa.TreeStep(k, v, ke, ve, batch=len(q), num_heads=H, max_seqlen_q=bound,
                         max_blocks_per_seq=c.batch.tables.shape[1])
    c.run()
    assert c.step.status() == (pa.PA_ERR_INVALID_ARG, pa.PA_STATUS_BIT_PLAN)
    live = np.repeat(c.batch.q <= bound, c.batch.q)
    c.check(live)
    assert (c.out[:c.tokens].cpu().numpy()[~live] == 7).all()


@pytest.mark.parametrize("shape", [(4, 2, 64), (8, 2, 128), (32, 4, 128), (2, 1, 272)], ids=str)
def test_lengths_whose_sum_passes_32_bits(torch, shape):
    """Sequences that state two thousand million tokens are left out, those before them are right,
    those behind them have no rows."""
    H, Hk, d = shape
    q = [3, 2, 1, 1, 1, 1, 4]
    c = Case(torch, 8, q, [30 + n for n in q], H, Hk, d, d, 16, "tree", behind=1)
    (k, ke), (v, ve) = c.dev
    c.step = pa.TreeStep(k, v, ke, ve, batch=len(q), num_heads=H, max_seqlen_q=8,
                         max_blocks_per_seq=c.batch.tables.shape[1])
    stated = c.batch.q.copy()
    stated[2:6] = 2**31 - 1
    c.args[3] = up(torch, stated)
    c.run()
    assert c.step.status() == (pa.PA_ERR_INVALID_ARG, pa.PA_STATUS_BIT_PLAN)
    c.check(np.arange(c.tokens) < 5)
    assert (c.out[5:] == 7).all()
    cache = empty_cache(torch, c.batch.num_blocks, 16, Hk, d, d)
    x = rows(np.random.default_rng(0), c.tokens, Hk, d)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache.write(up(torch, x), up(torch, x), c.args[1], c.args[2], c.args[3], 8, status=status)
    assert status.item() == pa.PA_STATUS_BIT_PLAN
    good = ref.Batch(c.batch.tables, c.batch.ctx, np.array([3, 2, 0, 0, 0, 0, 0]), 16, c.batch.num_blocks)
    want, want_e = expected_cache(good, x[:5], d, Hk)
    assert ref.same_codes(cache.key.view(torch.uint8).cpu().numpy(), want)
    np.testing.assert_array_equal(cache.key_exps.cpu().numpy(), want_e)


@pytest.mark.parametrize("call", ["write", "store"])
@pytest.mark.parametrize("fault", ["negative", "more than the tokens", "no lengths"])
def test_the_cache_reports_lengths_that_no_token_belongs_to(torch, call, fault):
    rng = np.random.default_rng(7)
    q = [1] * 5 if fault == "no lengths" else [2, 1, 3, 2, 1]
    batch = ref.make_batch(rng, q, [n + 20 for n in q], 16)
    stated, T, stored = batch.q.copy(), int(batch.q.sum()), np.array(q)
    if fault == "negative":
        stated[1], stored[1] = -3, 0
        T -= 1
    else:
        T -= 2  # the last sequence and a token of the one before it, or two sequences
        stored = np.array([1, 1, 1, 0, 0]) if fault == "no lengths" else np.array([2, 1, 3, 1, 0])
    k, v, xq = rows(rng, T, 2, 64), rows(rng, T, 2, 64), rows(rng, T, 4, 64)
    c = empty_cache(torch, batch.num_blocks, 16, 2, 64, 64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lens = (up(torch, batch.tables), up(torch, batch.ctx),
            None if fault == "no lengths" else up(torch, stated), 3)
    if call == "write":
        c.write(up(torch, k), up(torch, v), *lens, status=status)
    else:
        c.store(up(torch, xq), up(torch, k), up(torch, v), None, None, None, None, *lens,
                torch.zeros((T, 4, 64), dtype=torch.float16, device="cuda"), status=status)
    assert status.item() == pa.PA_STATUS_BIT_PLAN
    # the stored tokens of a sequence are its first ones
    ctx = batch.ctx - np.array(q) + stored if fault != "negative" else batch.ctx
    good = ref.Batch(batch.tables, ctx, stored, 16, batch.num_blocks)
    want, want_e = expected_cache(good, k, 64, 2)
    assert ref.same_codes(c.key.view(torch.uint8).cpu().numpy(), want)
    np.testing.assert_array_equal(c.key_exps.cpu().numpy(), want_e)


@pytest.mark.parametrize("shape", [(4, 2, 64), (32, 4, 128), (2, 1, 272)], ids=str)
@pytest.mark.parametrize("fault", ["negative", "more than the tokens", "context"])
def test_the_attention_reports_lengths_that_no_token_belongs_to(torch, shape, fault):
    H, Hk, d = shape
    q = [2, 0, 3, 2, 1]
    c = Case(torch, 8, q, [n + 20 for n in q], H, Hk, d, d, 16, "tree")
    stated, ctx, rows_in = c.batch.q.copy(), c.batch.ctx.copy(), c.tokens
    if fault == "negative":
        stated[1] = -1
    elif fault == "context":
        ctx[1] = -1  # of a sequence without tokens
    else:
        rows_in -= 2
    c.args[0], c.args[2], c.args[3] = c.args[0][:rows_in], up(torch, ctx), up(torch, stated)
    c.args[4], out = c.args[4][:rows_in].contiguous(), c.out
    c.out = out[:rows_in]
    c.run()
    assert c.step.status() == (pa.PA_ERR_INVALID_ARG, pa.PA_STATUS_BIT_PLAN)
    assert (out[rows_in:] == 7).all()
    want, bound = ref.tree_attention(c.query, *c.real, *c.exp, c.batch, c.parents, c.scale)
    got = out.cpu().numpy().astype(np.float64)
    assert (np.abs(got - want)[:rows_in] <= bound[:rows_in]).all()
