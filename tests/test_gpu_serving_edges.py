"""Serving calls at sizes that the other tests leave out: many rows of the row kernels, 2048 sequences,
blocks of more than 128 tokens, caches past 32-bit offsets, queries that are not numbers."""
import numpy as np
import pytest

import paged_kv_cache_206_gb300 as pa
from . import serving_ref as ref
from .test_gpu_cache import check_half, empty_cache, expected_cache, rows, table, up
from .test_gpu_tree import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    torch.cuda.set_device(0)
    return torch


# tokens of the sequences, Hk, hk, hv: rows by two and by four to a group of lanes (both batches of a
# warp), a row over all lanes and over two rounds of them
MANY = [([700, 3, 200], 32, 128, 128), ([500, 0, 600], 40, 64, 64), ([900, 1], 9, 80, 48), ([1300], 5, 256, 256),
        ([700, 60], 3, 576, 512), ([2500], 17, 16, 16)]


@pytest.mark.parametrize("case", MANY, ids=lambda c: str(c[1:]))
def test_write_many_rows(torch, case):
    q, Hk, hk, hv = case
    rng = np.random.default_rng(Hk)
    batch = ref.make_batch(rng, q, [n + 13 for n in q], 48)
    T = int(batch.q.sum())
    k, v = rows(rng, T, Hk, hk), rows(rng, T, Hk, hv)
    k[5, Hk - 1, 3], v[T - 2, Hk // 2, 0] = np.inf, np.nan
    c = empty_cache(torch, batch.num_blocks, 48, Hk, hk, hv)
    c.write(up(torch, k), up(torch, v), up(torch, batch.tables), up(torch, batch.ctx), up(torch, batch.q), max(q))
    for x, hs, codes, exps in ((k, hk, c.key, c.key_exps), (v, hv, c.value, c.value_exps)):
        want, want_e = expected_cache(batch, x, hs, Hk)
        assert ref.same_codes(codes.view(torch.uint8).cpu().numpy(), want)
        np.testing.assert_array_equal(exps.cpu().numpy(), want_e)


@pytest.mark.parametrize("case", MANY, ids=lambda c: str(c[1:]))
@pytest.mark.parametrize("inter", [False, True])
def test_store_many_rows(torch, case, inter):
    """Queries, keys and values as test_store checks them: the exponent that a maximum within its fp32
    error needs, elements within half a step of e4m3 and that error."""
    q, Hk, hk, hv = case
    rng = np.random.default_rng(Hk + 1)
    H = 3 * Hk
    batch = ref.make_batch(rng, q, [n + 13 for n in q], 48)
    T = int(batch.q.sum())
    xq, xk, v = rows(rng, T, H, hk), rows(rng, T, Hk, hk), rows(rng, T, Hk, hv)
    w = [(1 + 0.2 * rng.normal(size=hk)).astype(np.float16) for _ in range(2)]
    rot = hk // 32 * 16 or hk
    cs = table(rng, 3000, rot)
    pos = np.concatenate([np.arange(L - n, L) for n, L in zip(batch.q, batch.ctx)])
    c = empty_cache(torch, batch.num_blocks, 48, Hk, hk, hv)
    qo = torch.zeros((T, H, hk), dtype=torch.float16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.store(up(torch, xq), up(torch, xk), up(torch, v), up(torch, w[0]), up(torch, w[1]), up(torch, cs), None,
            up(torch, batch.tables), up(torch, batch.ctx), up(torch, batch.q), max(q), qo, eps=1e-5,
            interleaved=inter, status=status)
    assert status.item() == 0
    eps = np.float64(np.float32(1e-5))
    want, mag = ref.rotate(xq, w[0], cs, pos, eps, inter)
    check_half(qo.cpu().numpy(), want, ref.rotate_error(mag, hk))
    want_v, want_ve = expected_cache(batch, v, hv, Hk)
    assert ref.same_codes(c.value.view(torch.uint8).cpu().numpy(), want_v)
    np.testing.assert_array_equal(c.value_exps.cpu().numpy(), want_ve)
    want, mag = ref.rotate(xk, w[1], cs, pos, eps, inter)
    error = 1.001 * ref.rotate_error(mag, hk)
    codes, exps = c.key.view(torch.uint8).cpu().numpy(), c.key_exps.cpu().numpy()
    for b in range(len(q)):
        n, L, t0 = int(batch.q[b]), int(batch.ctx[b]), int(batch.starts[b])
        if n == 0:
            continue
        blk, off = batch.slots(b, L - n, L)
        e = exps[blk, :, off].astype(np.int64) - 127
        y, err = want[t0:t0 + n], error[t0:t0 + n]
        assert ((e >= ref.row_exponent(np.maximum(np.abs(y) - err, 0))) & (e <= ref.row_exponent(np.abs(y) + err))).all()
        held = ref.decode(codes[blk, off]) * 2.0 ** e[..., None]
        half_step = np.maximum(2.0**-4 * (np.abs(y) + err), 2.0**-10 * 2.0 ** e[..., None])
        assert (np.abs(held - y) <= half_step + err).all()


def test_2048_sequences(torch):
    rng = np.random.default_rng(0)
    q = rng.integers(0, 4, 2048)
    q[-1] = 3
    c = Case(torch, 8, q, q + rng.integers(0, 40, 2048) * (q > 0), 4, 2, 16, 16, 16, "tree", behind=3)
    c.run()
    assert c.step.status() == (pa.PA_OK, 0)
    c.check()
    x = rows(rng, c.tokens, 2, 16)
    cache = empty_cache(torch, c.batch.num_blocks, 16, 2, 16, 16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache.write(up(torch, x), up(torch, x), *c.args[1:4], 3, status=status)
    assert status.item() == 0
    want, want_e = expected_cache(c.batch, x, 16, 2)
    assert ref.same_codes(cache.key.view(torch.uint8).cpu().numpy(), want)
    np.testing.assert_array_equal(cache.value_exps.cpu().numpy(), want_e)


@pytest.mark.parametrize("bs", [144, 160, 272, 512, 1024])
@pytest.mark.parametrize("shape", [(4, 1, 128), (16, 1, 64), (32, 1, 128), (64, 1, 64), (200, 1, 128), (8, 2, 256)], ids=str)
@pytest.mark.parametrize("bits", [8, 16])
def test_blocks_of_more_than_128_tokens(torch, bits, shape, bs):
    H, Hk, d = shape
    c = Case(torch, bits, [1, 1, 1], [1, 700, bs + 3], H, Hk, d, d, bs, "chain")
    c.run()
    assert c.step.status() == (pa.PA_OK, 0)
    c.check()
    if bits == 8:
        x = rows(np.random.default_rng(bs), 3, Hk, d)
        cache = empty_cache(torch, c.batch.num_blocks, bs, Hk, d, d)
        cache.write(up(torch, x), up(torch, x), c.args[1], c.args[2])
        k, v = (torch.zeros((3, Hk, d), dtype=torch.float16, device="cuda") for _ in range(2))
        cache.read(c.args[1], c.args[2] - 1, c.args[2], up(torch, np.arange(3, dtype=np.int32)), 1, k, v)
        codes, e = ref.quantise(x.astype(np.float64))
        held = (ref.decode(codes) * 2.0 ** e[..., None].astype(np.float64)).astype(np.float16)
        np.testing.assert_array_equal(k.cpu().numpy(), held)
        np.testing.assert_array_equal(v.cpu().numpy(), held)


@pytest.mark.parametrize("shape", [(8, 2, 128, 2), (8, 2, 64, 4), (16, 1, 128, 6), (16, 1, 128, 12), (4, 2, 272, 2)], ids=str)
@pytest.mark.parametrize("bits", [8, 16])
def test_a_query_that_is_no_number_keeps_to_its_row(torch, bits, shape):
    H, Hk, d, q = shape
    c = Case(torch, bits, [q, 1, q], [300, 40, 170], H, Hk, d, d, 16, "tree")
    want = c.run().clone()
    hit = [(0, 1), (q - 1, H - 1), (q + 1, 0)]
    for n, (t, h) in enumerate(hit):
        c.args[0][t, h, 3 * n] = (float("nan"), float("inf"), float("-inf"))[n]
    got = c.run()
    assert c.step.status() == (pa.PA_OK, 0)
    for t, h in hit:
        assert not bool(got[t, h].isfinite().any())
        got[t, h] = want[t, h]
    assert torch.equal(got, want)


@pytest.mark.parametrize("bits", [8, 16])
def test_caches_past_32_bit_offsets(torch, bits):
    """Sequences at the far end of a cache of more than 2^32 elements (and exponents past 2^25): stored,
    read back and attended there with the same bits as in a small one."""
    Hk, H, d, bs, used = 8, 32, 128, 128, 40
    blocks = 2**32 // (bs * Hk * d) + 500
    g = torch.Generator(device="cuda").manual_seed(1)
    lens = np.array([900, 1400, 300], np.int32)
    tables = np.zeros((3, 12), np.int32)
    at = 0
    for b, n in enumerate(-(-lens // bs)):
        tables[b, :n] = at + np.arange(n)
        at += n
    x = [torch.randn((int(lens.sum()), Hk, d), generator=g, device="cuda").half() for _ in range(2)]
    kinds = []
    for nb, shift in ((used, 0), (blocks, blocks - used)):
        t, n = up(torch, tables + shift), up(torch, lens)
        if bits == 8:
            parts = [torch.empty((nb, bs, Hk, d), dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
            parts += [torch.empty((nb, Hk, bs), dtype=torch.uint8, device="cuda") for _ in range(2)]
            cache = pa.QuantCache(*parts)
            cache.write(*x, t, n, n, int(lens.max()))
            back = [torch.zeros((int(lens.sum()), Hk, d), dtype=torch.float16, device="cuda") for _ in range(2)]
            cache.read(t, None, n, up(torch, np.array([0, 900, 2300], np.int32)), int(lens.max()), *back)
        else:
            parts, back = [torch.empty((nb, bs, Hk, d), dtype=torch.float16, device="cuda") for _ in range(2)], []
            for b in range(3):
                for p, rows_ in zip(parts, x):
                    first = int(lens[:b].sum())
                    for j in range(-(-int(lens[b]) // bs)):
                        piece = rows_[first + j * bs:first + min((j + 1) * bs, int(lens[b]))]
                        p[int(tables[b, j]) + shift, :len(piece)] = piece
            parts += [None, None]
        outs = []
        for q in (1, 4, 30, 70):
            query = torch.randn((3 * q, H, d), generator=torch.Generator(device="cuda").manual_seed(q),
                                device="cuda").half()
            step = pa.TreeStep(*parts, batch=3, num_heads=H, max_seqlen_q=q, max_blocks_per_seq=12)
            outs.append(step.run(query, t, n, up(torch, np.full(3, q, np.int32)), None, torch.empty_like(query)))
            assert step.status() == (pa.PA_OK, 0)
        kinds.append(back + outs)
        del parts
        torch.cuda.empty_cache()
    for small, far in zip(*kinds):
        assert torch.equal(small, far) and bool(small.isfinite().all())


def test_two_threads_at_once(torch):
    """A thread that attends and one that reads the same 8-bit cache back, each on a stream of its own and
    with configurations that change from call to call."""
    import threading

    from paged_kv_cache_206_gb300 import serving
    c = Case(torch, 8, [4] * 6, [500, 30, 900, 4, 77, 260], 8, 2, 128, 128, 16, "tree")
    (k, ke), (v, ve) = c.dev
    cache = pa.QuantCache(k, v, ke, ve)
    n = int(c.batch.ctx.sum())
    at = up(torch, (np.cumsum(c.batch.ctx) - c.batch.ctx).astype(np.int32))
    kv = [torch.zeros((n, 2, 128), dtype=torch.float16, device="cuda") for _ in range(2)]
    want = c.run().clone()
    cache.read(c.args[1], None, c.args[2], at, 900, *kv)
    held = [t.clone() for t in kv]
    torch.cuda.synchronize()
    wrong, streams = [], [torch.cuda.Stream() for _ in range(2)]

    def attend():
        with torch.cuda.stream(streams[0]):
            for _ in range(300):
                if not torch.equal(c.run(), want):
                    wrong.append("attention")

    def read():
        with torch.cuda.stream(streams[1]):
            for i in range(300):
                cache.read(c.args[1], None, c.args[2], at, 900 + i, *kv)
                cache._configs.clear()
                serving._rotations.clear()
                if not all(torch.equal(a, b) for a, b in zip(kv, held)):
                    wrong.append("read")
    def kept(f):
        try:
            f()
        except Exception as e:  # a thread's own exception ends no test
            wrong.append(e)
    threads = [threading.Thread(target=kept, args=(f,)) for f in (attend, read)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong


@pytest.mark.parametrize("call", [(8, 2, 64, 2), (8, 2, 256, 2), (16, 1, 128, 6), (4, 2, 272, 2), "forward"], ids=str)
def test_a_threads_first_cuda_call(torch, call):
    """In a thread that has called nothing of CUDA before."""
    import threading
    if call == "forward":
        from paged_kv_cache_206_gb300 import workloads as W
        db = pa.DeviceBatch(W.gqa_decode(batch=3, max_len=500, seed=77))
        run, status = db.forward, db.status
    else:
        H, Hk, d, q = call
        c = Case(torch, 8, [q, 1], [300, 40], H, Hk, d, d, 16, "tree")
        run, status = c.run, c.step.status
    torch.cuda.synchronize()
    failed = []

    def first():
        try:
            run()
        except Exception as e:
            failed.append(e)
    t = threading.Thread(target=first)
    t.start()
    t.join()
    assert not failed and status() == (pa.PA_OK, 0), failed
    got = (db.out if call == "forward" else c.out).clone()
    assert torch.equal(run(), got)
