"""pa_qk_norm_rope, pa_cache_write, pa_cache_store and pa_cache_read on the GPU
against the 64-bit references."""
import numpy as np
import pytest

import paged_kv_cache_206_gb300 as pa
from . import serving_ref as ref

pytestmark = pytest.mark.gpu

SENTINEL = 0x5A


@pytest.fixture(scope="module")
def torch():
    import torch
    torch.cuda.set_device(0)
    return torch


def up(torch, a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def table(rng, rows, rot):
    freq = 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
    angle = np.arange(rows)[:, None] * freq
    return np.concatenate([np.cos(angle), np.sin(angle)], 1).astype(np.float32)


def rows(rng, *shape):
    """Rows of several magnitudes, with a zero row and a tiny one."""
    x = rng.normal(size=shape) * 2.0 ** rng.integers(-6, 7, shape[:2])[..., None]
    x = x.astype(np.float16)
    x[0, 0] = 0
    x[-1, -1] *= np.float16(2.0**-12)
    return x


def check_half(got, want, error):
    """Half a step of fp16 of the value (2^-11 relative, 2^-25 absolute) and the fp32 error."""
    want = np.asarray(want)
    with np.errstate(invalid="ignore"):
        ok = np.abs(got.astype(np.float64) - want) <= 2.0**-11 * np.abs(want) + 1.001 * error + 2.0**-25
    assert ok.all(), np.argwhere(~ok)[:5]


# tokens, H, Hk, hk, rotary dim, interleaved, norm of q, of k, packed projection
ROTATE = [
    (1, 32, 8, 128, 128, False, True, True, True),
    (1, 1, 1, 16, 16, True, True, False, False),
    (7, 4, 2, 64, 32, False, True, True, True),
    (33, 28, 4, 128, 64, True, False, True, False),
    (5, 6, 3, 256, 256, False, True, True, True),
    (19, 3, 1, 576, 64, True, True, True, True),
    (4, 2, 2, 576, 576, False, False, False, False),
    (130, 40, 40, 48, 48, False, True, True, True),
    (9, 5, 7, 80, 0, False, True, True, True),
    (300, 8, 2, 512, 128, True, True, True, False),
    (1000, 32, 8, 128, 128, False, True, True, True),
]


@pytest.mark.parametrize("case", ROTATE, ids=str)
def test_rotate(torch, case):
    tokens, H, Hk, hk, rot, inter, nq, nk, packed = case
    rng = np.random.default_rng(tokens * 7 + H)
    x = rows(rng, tokens, H + 2 * Hk, hk)
    w = [(1 + 0.2 * rng.normal(size=hk)).astype(np.float16) if on else None for on in (nq, nk)]
    cs = table(rng, 50, rot) if rot else None
    pos = rng.integers(0, 50, tokens).astype(np.int32)
    pos[tokens // 2] = -1 if tokens > 3 else pos[tokens // 2]
    d = up(torch, x)
    q, k = d[:, :H], d[:, H:H + Hk]
    if not packed:
        q, k = q.contiguous(), k.contiguous()
    qo = torch.full((tokens, H, hk), 7.0, dtype=torch.float16, device="cuda")
    ko = torch.full((tokens, Hk, hk), 7.0, dtype=torch.float16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_qk_norm_rope(q, k, up(torch, w[0]), up(torch, w[1]), up(torch, cs), up(torch, pos), qo, ko,
                       eps=1e-5, interleaved=inter, status=status)
    assert status.item() == 0
    live = pos >= 0
    for got, part, weight in ((qo, x[:, :H], w[0]), (ko, x[:, H:H + Hk], w[1])):
        got = got.cpu().numpy()
        want, mag = ref.rotate(part[live], weight, cs, pos[live], np.float64(np.float32(1e-5)), inter)
        check_half(got[live], want, ref.rotate_error(mag, hk))
        assert (got[~live] == 7).all()


def test_rotate_in_place_and_bad_positions(torch):
    rng = np.random.default_rng(5)
    q, k = rows(rng, 6, 4, 64), rows(rng, 6, 2, 64)
    cs, pos = table(rng, 10, 64), np.array([0, 9, 10, -2, -1, 3], np.int32)
    dq, dk, w = up(torch, q), up(torch, k), up(torch, np.ones(64, np.float16))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_qk_norm_rope(dq, dk, w, w, up(torch, cs), up(torch, pos), dq, dk, status=status)
    assert status.item() == pa.PA_STATUS_BIT_POSITION
    assert pa.pa_status_read(status)[0] == pa.PA_ERR_INVALID_ARG
    live = (pos >= 0) & (pos < 10)
    for got, part in ((dq, q), (dk, k)):
        got = got.cpu().numpy()
        want, mag = ref.rotate(part[live], np.ones(64, np.float16), cs, pos[live],
                               np.float64(np.float32(1e-6)), False)
        check_half(got[live], want, ref.rotate_error(mag, 64))
        np.testing.assert_array_equal(got[~live], part[~live])


def test_rotate_keeps_nan_to_its_row(torch):
    x = np.ones((3, 4, 64), np.float16)
    x[1, 2, 5], x[2, 0, 9] = np.nan, np.inf
    cs, w = table(None, 4, 64), up(torch, np.ones(64, np.float16))
    d, pos = up(torch, x), torch.zeros(3, dtype=torch.int32, device="cuda")
    qo, ko = torch.empty_like(d[:, :2]).contiguous(), torch.empty_like(d[:, 2:]).contiguous()
    pa.pa_qk_norm_rope(d[:, :2], d[:, 2:], w, w, up(torch, cs), pos, qo, ko)
    bad = np.isnan(np.concatenate([qo.cpu().numpy(), ko.cpu().numpy()], 1)).any(-1)
    want = np.zeros((3, 4), bool)
    want[1, 2] = want[2, 0] = True
    np.testing.assert_array_equal(bad, want)


def empty_cache(torch, nb, bs, Hk, hk, hv):
    c = pa.QuantCache.empty(nb, bs, Hk, hk, hv)
    for t in (c.key, c.value, c.key_exps, c.value_exps):
        t.view(torch.uint8).fill_(SENTINEL)
    return c


def expected_cache(batch, x, hs, Hk, lead=0):
    """Codes and exponents after the rows x [T, Hk, hs] were written."""
    codes = np.full((batch.num_blocks, batch.block, Hk, hs), SENTINEL, np.uint8)
    exps = np.full((batch.num_blocks, Hk, batch.block), SENTINEL, np.uint8)
    with np.errstate(invalid="ignore"):  # signalling NaN
        x = x.astype(np.float64)
    qc, qe = ref.quantise(x)
    for b in range(len(batch.q)):
        n, L, t0 = int(batch.q[b]), int(batch.ctx[b]), int(batch.starts[b])
        blk, off = batch.slots(b, L - n, L)
        codes[blk, off] = qc[t0:t0 + n]
        exps[blk, :, off] = qe[t0:t0 + n] + 127
    return codes, exps


# q, ctx, Hk, hk, hv, block size
WRITE = [
    ([1], [1], 1, 16, 16, 16),
    ([1, 1, 1], [5, 16, 17], 8, 128, 128, 16),
    ([3, 0, 16, 1], [3, 9, 40, 33], 2, 64, 64, 16),
    ([130], [300], 4, 128, 128, 128),
    ([2, 5], [2, 70], 3, 576, 512, 64),
    ([7, 1], [48, 49], 5, 80, 48, 48),
    ([1] * 40, list(range(1, 41)), 2, 256, 256, 32),
    ([0, 0, 6], [0, 20, 6], 2, 576, 16, 16),
]


@pytest.mark.parametrize("case", WRITE, ids=str)
@pytest.mark.parametrize("lens", ["given", "default"])
def test_write(torch, case, lens):
    q, ctx, Hk, hk, hv, bs = case
    if lens == "default" and set(q) != {1}:
        pytest.skip("q_seqlens may be left out only when every q is 1")
    rng = np.random.default_rng(len(q) + hk)
    batch = ref.make_batch(rng, q, ctx, bs)
    T, behind = int(batch.q.sum()), 3 if lens == "given" else 0
    k, v = rows(rng, T + behind, Hk, hk), rows(rng, T + behind, Hk, hv)
    if T > 2:
        k[1, 0, 3], k[2, -1, 0], v[1, 0, 7] = np.nan, -np.inf, np.inf
        v[2, 0] = np.nan
    c = empty_cache(torch, batch.num_blocks, bs, Hk, hk, hv)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.write(up(torch, k), up(torch, v), up(torch, batch.tables), up(torch, batch.ctx),
            up(torch, batch.q) if lens == "given" else None, max(q), status=status)
    assert status.item() == 0
    for x, hs, codes, exps in ((k, hk, c.key, c.key_exps), (v, hv, c.value, c.value_exps)):
        want, want_e = expected_cache(batch, x, hs, Hk)
        assert ref.same_codes(codes.view(torch.uint8).cpu().numpy(), want)
        np.testing.assert_array_equal(exps.cpu().numpy(), want_e)


def test_every_half_is_held_as_defined(torch):
    """All fp16 bit patterns, 64 to a row of neighbours and 64 to a row of strangers."""
    x = np.arange(65536, dtype=np.uint16).view(np.float16)
    x = np.concatenate([x.reshape(1024, 1, 64), np.random.default_rng(1).permutation(x).reshape(1024, 1, 64)])
    batch = ref.make_batch(np.random.default_rng(0), [2048], [2048], 128)
    c = empty_cache(torch, batch.num_blocks, 128, 1, 64, 64)
    d = up(torch, x)
    c.write(d, d, up(torch, batch.tables), up(torch, batch.ctx), up(torch, batch.q), 2048)
    want, want_e = expected_cache(batch, x, 64, 1)
    for codes, exps in ((c.key, c.key_exps), (c.value, c.value_exps)):
        assert ref.same_codes(codes.view(torch.uint8).cpu().numpy(), want)
        np.testing.assert_array_equal(exps.cpu().numpy(), want_e)


STORE = [
    ([1, 1], [1, 40], 32, 8, 128, 128, 128, False, True, True),
    ([5, 0, 9], [5, 7, 90], 4, 2, 64, 64, 32, True, True, False),
    ([64], [64], 28, 4, 128, 64, 128, False, True, True),
    ([3, 2], [17, 2], 2, 1, 576, 512, 64, True, False, True),
    ([1, 4, 2], [16, 33, 64], 6, 3, 256, 256, 256, False, True, False),
]


@pytest.mark.parametrize("case", STORE, ids=str)
def test_store(torch, case):
    q, ctx, H, Hk, hk, hv, rot, inter, norm, given = case
    rng = np.random.default_rng(hk + H)
    batch = ref.make_batch(rng, q, ctx, 16)
    T = int(batch.q.sum())
    xq, xk, v = rows(rng, T, H, hk), rows(rng, T, Hk, hk), rows(rng, T, Hk, hv)
    w = [(1 + 0.2 * rng.normal(size=hk)).astype(np.float16) if norm else None for _ in range(2)]
    cs = table(rng, 128, rot)
    pos = np.concatenate([np.arange(L - n, L) for n, L in zip(q, ctx)]).astype(np.int32)
    if given:
        pos = rng.integers(0, 128, T).astype(np.int32)
    c = empty_cache(torch, batch.num_blocks, 16, Hk, hk, hv)
    qo = torch.zeros((T, H, hk), dtype=torch.float16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if hk == hv:  # one packed projection
        d = up(torch, np.concatenate([xq, xk, v], 1))
        dq, dk, dv = d[:, :H], d[:, H:H + Hk], d[:, H + Hk:]
    else:
        dq, dk, dv = up(torch, xq), up(torch, xk), up(torch, v)
    c.store(dq, dk, dv, up(torch, w[0]), up(torch, w[1]), up(torch, cs),
            up(torch, pos) if given else None, up(torch, batch.tables), up(torch, batch.ctx),
            up(torch, batch.q), max(q), qo, eps=1e-5, interleaved=inter, status=status)
    assert status.item() == 0
    eps = np.float64(np.float32(1e-5))
    want, mag = ref.rotate(xq, w[0], cs, pos, eps, inter)
    check_half(qo.cpu().numpy(), want, ref.rotate_error(mag, hk))
    want_v, want_ve = expected_cache(batch, v, hv, Hk)
    assert ref.same_codes(c.value.view(torch.uint8).cpu().numpy(), want_v)
    np.testing.assert_array_equal(c.value_exps.cpu().numpy(), want_ve)
    # keys: the exponent that a maximum within its fp32 error needs, and every
    # element within half a step of e4m3 and that error
    want, mag = ref.rotate(xk, w[1], cs, pos, eps, inter)
    error = 1.001 * ref.rotate_error(mag, hk)
    codes = c.key.view(torch.uint8).cpu().numpy()
    exps = c.key_exps.cpu().numpy()
    touched = np.zeros(exps.shape, bool)
    for b in range(len(q)):
        n, L, t0 = q[b], ctx[b], int(batch.starts[b])
        blk, off = batch.slots(b, L - n, L)
        e = exps[blk, :, off].astype(np.int64) - 127
        touched[blk, :, off] = True
        y, err = want[t0:t0 + n], error[t0:t0 + n]
        lo = ref.row_exponent(np.maximum(np.abs(y) - err, 0))
        hi = ref.row_exponent(np.abs(y) + err)
        assert ((e >= lo) & (e <= hi)).all()
        held = ref.decode(codes[blk, off]) * 2.0 ** e[..., None]
        half_step = np.maximum(2.0**-4 * (np.abs(y) + err), 2.0**-10 * 2.0 ** e[..., None])
        assert (np.abs(held - y) <= half_step + err).all()
    assert (exps[~touched] == SENTINEL).all()
    assert (codes.transpose(0, 2, 1, 3)[~touched] == SENTINEL).all()


def test_write_leaves_out_what_is_wrong(torch):
    """Bad lengths, bad blocks and bad positions: only the good tokens are stored."""
    rng = np.random.default_rng(2)
    batch = ref.make_batch(rng, [2, 2, 2, 2], [20, 5, 30, 12], 16)
    Hk, hk = 2, 64
    k, v = rows(rng, 8, Hk, hk), rows(rng, 8, Hk, hk)
    tables, ctx = batch.tables.copy(), batch.ctx.copy()
    ctx[1] = 1            # fewer than its current tokens
    ctx[3] = 10_000       # past the block table's row
    tables[2, 1] = batch.num_blocks  # the block of positions 28 and 29
    c = empty_cache(torch, batch.num_blocks, 16, Hk, hk, hk)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.write(up(torch, k), up(torch, v), up(torch, tables), up(torch, ctx), up(torch, batch.q), 2,
            status=status)
    assert status.item() == pa.PA_STATUS_BIT_PLAN | pa.PA_STATUS_BIT_BLOCK_INDEX
    good = ref.Batch(batch.tables, np.array([20, 0, 0, 0]), np.array([2, 0, 0, 0]), 16, batch.num_blocks)
    want, want_e = expected_cache(good, k, hk, Hk)
    assert ref.same_codes(c.key.view(torch.uint8).cpu().numpy(), want)
    np.testing.assert_array_equal(c.key_exps.cpu().numpy(), want_e)


# ctx, starts, Hk, hk, hv, block
READ = [
    ([1], None, 1, 16, 16, 16),
    ([37], None, 8, 128, 128, 16),
    ([0, 5, 100, 64], [0, 5, 3, 63], 3, 64, 80, 32),
    ([300, 1, 129], None, 2, 576, 512, 128),
    ([33, 47, 48, 95, 96], [1, 0, 2, 90, 95], 5, 48, 256, 48),
    ([2000, 700], [17, 0], 4, 256, 256, 64),
]


@pytest.mark.parametrize("case", READ, ids=str)
def test_read(torch, case):
    ctx, starts, Hk, hk, hv, bs = case
    rng = np.random.default_rng(sum(ctx))
    batch = ref.make_batch(rng, [0] * len(ctx), ctx, bs)
    st = np.zeros(len(ctx), np.int32) if starts is None else np.asarray(starts, np.int32)
    counts = batch.ctx - st
    out_starts = (np.cumsum(counts) - counts + 2).astype(np.int32)
    n = int(counts.sum()) + 5
    c = pa.QuantCache.empty(batch.num_blocks, bs, Hk, hk, hv)
    outs, parts = [], []
    for codes, exps, hs in ((c.key, c.key_exps, hk), (c.value, c.value_exps, hv)):
        hc = rng.integers(0, 256, codes.shape).astype(np.uint8)  # NaN codes among them
        he = rng.integers(95, 141, exps.shape).astype(np.uint8)
        codes.view(torch.uint8).copy_(up(torch, hc))
        exps.copy_(up(torch, he))
        outs.append(torch.full((n, Hk, hs), 7.0, dtype=torch.float16, device="cuda"))
        parts.append((hc, he))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.read(up(torch, batch.tables), up(torch, st) if starts is not None else None, up(torch, batch.ctx),
           up(torch, out_starts), int(counts.max()), *outs, status=status)
    assert status.item() == 0
    for got, (hc, he) in zip(outs, parts):
        want = np.full(got.shape, 7.0, np.float16)
        for b in range(len(ctx)):
            blk, off = batch.slots(b, int(st[b]), int(batch.ctx[b]))
            held = ref.decode(hc[blk, off]) * 2.0 ** (he[blk, :, off].astype(np.float64) - 127)[..., None]
            with np.errstate(over="ignore"):
                want[out_starts[b]:out_starts[b] + counts[b]] = held.astype(np.float16)
        np.testing.assert_array_equal(got.cpu().numpy(), want)


def test_read_leaves_out_what_is_wrong(torch):
    batch = ref.make_batch(np.random.default_rng(3), [0] * 5, [20, 8, 10, 6, 7], 16)
    c = pa.QuantCache.empty(batch.num_blocks, 16, 2, 64)
    c.key.view(torch.uint8).fill_(0x38)  # 1.0
    c.key_exps.fill_(127)
    tables, ctx, st = batch.tables.copy(), batch.ctx.copy(), np.zeros(5, np.int32)
    tables[0, 1] = -1        # positions 16..19
    st[1] = 9                # past its end
    ctx[2] = 30              # more rows than max_rows, and than the table's blocks
    out_starts = np.array([0, 20, 28, 35, 60], np.int32)  # 35..40 hits the end of the rows
    k = torch.full((38, 2, 64), 7.0, dtype=torch.float16, device="cuda")
    v = torch.full_like(k, 7.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.read(up(torch, tables), up(torch, st), up(torch, ctx), up(torch, out_starts), 20, k, v, status=status)
    assert status.item() == (pa.PA_STATUS_BIT_PLAN | pa.PA_STATUS_BIT_BLOCK_INDEX
                             | pa.PA_STATUS_BIT_WORKSPACE)
    want = np.full(38, 7.0)
    want[0:16] = 1
    want[35:38] = 1
    np.testing.assert_array_equal(k.cpu().numpy()[:, 0, 0], want)
    np.testing.assert_array_equal((v == 7).cpu().numpy()[:, 1, 63], want == 7)
