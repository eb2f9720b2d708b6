"""Waits of the kernels of pa_window_forward that run out, without a GPU fault: with a limit of a few
cycles a correct launch must report PA_ERR_TIMEOUT, exit with its copies landed and its tensor memory
freed, and leave the context usable: with the default limit back the same call gives the same bits.
And batches at the ends of what the call takes."""
import numpy as np
import pytest

import paged_kv_cache_206_gb300 as pa
from . import serving_ref as ref
from .test_gpu_window import Case, up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    torch.cuda.set_device(0)
    yield torch
    pa.testing_set_wait_limit(0)


# tokens, H, Hk, dims, window: few rows of a kv head, up to 128, more; a group that is no power of two
LIMITS = [(1, 32, 8, 128, 3000), (4, 32, 8, 128, 3000), (2, 16, 4, 256, 3000), (16, 32, 8, 128, 2000),
          (16, 32, 8, 64, 2000), (300, 32, 8, 128, 500), (300, 32, 8, 64, 500), (300, 28, 4, 128, 500)]


@pytest.mark.parametrize("case", LIMITS, ids=str)
@pytest.mark.parametrize("bits", [8, 16])
def test_short_wait_limit_times_out_and_the_context_survives(torch, bits, case):
    tokens, H, Hk, d, window = case
    B, bs = 24, 64
    rng = np.random.default_rng(tokens)
    g = torch.Generator(device="cuda").manual_seed(tokens)
    q = rng.integers(max(1, tokens // 2), tokens + 1, B).astype(np.int32)
    ctx = np.maximum(q, rng.integers(64, 6000, B)).astype(np.int32)
    batch = ref.make_batch(rng, q, ctx, bs)
    k, v = (torch.randn((batch.num_blocks, bs, Hk, d), generator=g, device="cuda").half() for _ in range(2))
    exps = [None, None]
    if bits == 8:
        k, v = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)
        exps = [torch.randint(125, 129, (batch.num_blocks, Hk, bs), generator=g, device="cuda").to(torch.uint8)
                for _ in range(2)]
    query = torch.randn((int(q.sum()), H, d), generator=g, device="cuda").half()
    step = pa.WindowStep(k, v, *exps, batch=B, num_heads=H, max_seqlen_q=tokens,
                         max_blocks_per_seq=batch.tables.shape[1], window=window, sinks=4)
    args = (query, up(torch, batch.tables), up(torch, ctx), up(torch, q), torch.empty_like(query))
    flush = torch.empty(512 << 20, dtype=torch.uint8, device="cuda")
    first = step.run(*args).clone()
    assert step.status() == (pa.PA_OK, 0)
    # whether a wait outlasts 32 cycles depends on when its copy lands: from HBM, in three tries
    for _ in range(3):
        flush.zero_()
        pa.testing_set_wait_limit(32)
        try:
            step.run(*args)
            st, word = step.status()
        finally:
            pa.testing_set_wait_limit(0)
        if st == pa.PA_ERR_TIMEOUT:
            break
    assert st == pa.PA_ERR_TIMEOUT and word == pa.PA_STATUS_BIT_TIMEOUT
    pa.pa_status_clear(step.workspace)
    for _ in range(3):
        assert torch.equal(step.run(*args), first)
    assert step.status() == (pa.PA_OK, 0)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("q,H,Hk,d,window,sinks", [(1, 8, 2, 128, 15000, 4), (1, 8, 2, 64, 700, 5000),
                                                   (100, 2, 1, 128, 15000, 300), (9, 8, 2, 128, 30000, 0),
                                                   (400, 2, 2, 64, 9000, 4)])
def test_one_long_sequence_on_all_workers(torch, bits, q, H, Hk, d, window, sinks):
    c = Case(torch, bits, [q], [20000 + q], H, Hk, d, d, 128, window, sinks)
    c.run()
    assert c.step.status() == (pa.PA_OK, 0)
    c.check()


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("drafts", [1, 3, 40])
def test_the_most_sequences(torch, bits, drafts):
    """2048 sequences, every third one padding."""
    rng = np.random.default_rng(drafts)
    q = rng.integers(1, drafts + 1, 2048) * (np.arange(2048) % 3 != 1)
    c = Case(torch, bits, q, q + rng.integers(0, 90, 2048), 4, 1, 64, 64, 16, 30, 3)
    c.run()
    assert c.step.status() == (pa.PA_OK, 0)
    c.check(list(range(0, 2048, 31)) + [2047])


@pytest.mark.parametrize("max_q", [1, 4, 64, 500])
def test_nothing_to_attend(torch, max_q):
    """A batch of padding alone, with rows that belong to nobody, and no rows at all."""
    c = Case(torch, 16, [0, 0, 0], [0, 40, 7], 8, 2, 128, 128, 16, 20, 2, behind=5, max_q=max_q)
    c.run()
    assert c.step.status() == (pa.PA_OK, 0) and bool((c.out == 7).all())
    empty = c.args[0][:0]
    assert c.step.run(empty, *c.args[1:], c.out[:0]).numel() == 0


def test_rows_beyond_the_sequences_are_left_in_captured_batches(torch):
    """A graph of a full batch, replayed with fewer tokens in it: the other rows stay as they are."""
    for bits, q in ((8, 2), (16, 70)):
        c = Case(torch, bits, [q] * 5, [q + 200] * 5, 8, 2, 128, 128, 16, 64, 4)
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        c.run(stream=s)
        s.synchronize()
        with torch.cuda.graph(g, stream=s):
            c.run()
        c.args[3].copy_(up(torch, np.array([q, 0, q, 0, 0], np.int32)))
        c.out.fill_(7)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert bool((c.out[2 * q:] == 7).all()) and not bool((c.out[:2 * q] == 7).all(-1).any())
        assert c.step.status() == (pa.PA_OK, 0)


LONGEST = 2**31 - 4096


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("q,H,Hk,d", [(1, 8, 2, 128), (5, 8, 2, 64), (60, 4, 2, 128), (200, 4, 1, 64), (2, 4, 2, 320)])
def test_the_longest_context(torch, bits, q, H, Hk, d):
    """The keys of a short sequence at the two ends of the longest one, whose table has blocks nowhere
    else; one key more is refused."""
    bs, short = 128, 640
    c = Case(torch, bits, [q], [short], H, Hk, d, d, bs, 200, 20)
    tables = torch.full((1, 2**31 // bs), -1, dtype=torch.int32, device="cuda")
    tables[0, 0] = c.args[1][0, 0]
    tables[0, (LONGEST - short) // bs + 1:LONGEST // bs] = c.args[1][0, 1:short // bs]
    (k, ke), (v, ve) = c.dev
    c.step = pa.WindowStep(k, v, ke, ve, batch=1, num_heads=H, max_seqlen_q=q, max_blocks_per_seq=tables.shape[1],
                           window=200, sinks=20)
    c.args[1:3] = tables, torch.tensor([LONGEST + 1], dtype=torch.int32, device="cuda")
    c.run()
    assert c.step.status() == (pa.PA_ERR_INVALID_ARG, pa.PA_STATUS_BIT_PLAN)
    assert bool((c.out == 7).all())
    tree = pa.TreeStep(k, v, ke, ve, batch=1, num_heads=H, max_seqlen_q=q, max_blocks_per_seq=tables.shape[1])
    tree.run(*c.args, None, c.out)
    assert tree.status() == (pa.PA_ERR_INVALID_ARG, pa.PA_STATUS_BIT_PLAN)
    assert bool((c.out == 7).all())
    pa.pa_status_clear(c.step.workspace)
    c.args[2].fill_(LONGEST)
    c.run()
    assert c.step.status() == (pa.PA_OK, 0)
    c.check()


@pytest.mark.parametrize("q", [1, 40, 200])
def test_all_keys_of_the_longest_context(torch, q):
    """Keys of zero, so that every weight is the same, values of 1 in three quarters of the blocks and
    -1 in the others. A worker's sums are of whole numbers below 2^24 (a power of two's multiples), so
    only the join of at most 1216 parts (half a step each in the sums of weights and of values) and the
    result's rounding are off: 2 * 1216 * 2^-24 + 2^-12 < 4e-4 of 1/2 to 1."""
    bs, nb, d = 128, 512, 64
    cols, ones = 2**31 // bs, LONGEST // bs * 3 // 4
    g = torch.Generator(device="cuda").manual_seed(q)
    key = torch.zeros((nb, bs, 1, d), device="cuda").to(torch.float8_e4m3fn)
    value = torch.ones((nb, bs, 1, d), device="cuda")
    value[nb // 2:] = -1
    exps = [torch.full((nb, 1, bs), 127, dtype=torch.uint8, device="cuda") for _ in range(2)]
    tables = torch.randint(0, nb // 2, (1, cols), generator=g, device="cuda", dtype=torch.int32)
    tables[0, ones:] += nb // 2
    step = pa.WindowStep(key, value.to(torch.float8_e4m3fn), *exps, batch=1, num_heads=1, max_seqlen_q=q,
                         max_blocks_per_seq=cols, window=2**31 - 1)
    out = torch.full((q, 1, d), 7.0, dtype=torch.float16, device="cuda")
    step.run(torch.ones((q, 1, d), dtype=torch.float16, device="cuda"), tables,
             torch.tensor([LONGEST], dtype=torch.int32, device="cuda"),
             torch.tensor([q], dtype=torch.int32, device="cuda"), out)
    assert step.status() == (pa.PA_OK, 0)
    seen = LONGEST - q + 1 + np.arange(q)
    want = (2.0 * ones * bs - seen) / seen
    assert np.abs(out.cpu().numpy()[:, 0].astype(np.float64) - want[:, None]).max() < 4e-4
