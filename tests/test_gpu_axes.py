"""Rotation by positions of several axes, into fp16 rows and into the 8-bit cache, against the
64-bit reference."""
import numpy as np
import pytest

import paged_kv_cache_206_gb300 as pa
from . import serving_ref as ref
from . import window_ref as wref
from .test_gpu_cache import check_half, empty_cache, expected_cache, rows, table, up

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    torch.cuda.set_device(0)
    return torch


# tokens, H, Hk, hk, rotary dim, sections, cyclic, interleaved, norm, packed
CASES = [
    (1, 32, 8, 128, 128, (16, 24, 24), False, False, True, True),
    (1, 1, 1, 16, 16, (3, 3, 2), True, False, True, False),
    (33, 4, 2, 64, 32, (6, 5, 5), True, True, False, True),
    (7, 28, 4, 128, 64, (32,), False, False, True, True),
    (19, 6, 3, 256, 256, (100, 3, 25), False, True, True, True),
    (40, 3, 1, 576, 576, (99, 95, 94), True, False, True, True),
    (12, 2, 2, 576, 64, (0, 1, 31), False, False, True, True),
    (130, 5, 7, 80, 48, (6, 6, 6, 6), True, False, True, False),
    (9, 8, 2, 128, 128, (64, 0), False, True, True, True),
    (300, 40, 40, 64, 64, (30, 0, 2), True, False, False, False),
    (1000, 32, 8, 128, 128, (24, 20, 20), True, False, True, True),
    (1000, 32, 8, 128, 128, (16, 24, 24), False, True, True, True),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_rotate(torch, case):
    tokens, H, Hk, hk, rot, sections, cyclic, inter, norm, packed = case
    rng = np.random.default_rng(tokens + H)
    x = rows(rng, tokens, H + 2 * Hk, hk)
    w = [(1 + 0.2 * rng.normal(size=hk)).astype(np.float16) if norm else None for _ in range(2)]
    cs, pos = table(rng, 50, rot), rng.integers(0, 50, (len(sections), tokens)).astype(np.int32)
    if tokens > 3:
        pos[-1, tokens // 2] = -1
    d = up(torch, x)
    q, k = d[:, :H], d[:, H:H + Hk]
    if not packed:
        q, k = q.contiguous(), k.contiguous()
    qo = torch.full((tokens, H, hk), 7.0, dtype=torch.float16, device="cuda")
    ko = torch.full((tokens, Hk, hk), 7.0, dtype=torch.float16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_qk_norm_rope(q, k, up(torch, w[0]), up(torch, w[1]), up(torch, cs), up(torch, pos), qo, ko, eps=1e-5,
                       interleaved=inter, status=status, sections=sections, cyclic=cyclic)
    assert status.item() == 0
    live = (pos >= 0).all(0)
    for got, part, weight in ((qo, x[:, :H], w[0]), (ko, x[:, H:H + Hk], w[1])):
        got = got.cpu().numpy()
        want, mag = wref.rotate_axes(part[live], weight, cs, pos[:, live], sections, cyclic,
                                     np.float64(np.float32(1e-5)), inter)
        check_half(got[live], want, ref.rotate_error(mag, hk))
        assert (got[~live] == 7).all()


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("tokens", [1, 700])
@pytest.mark.parametrize("sections,cyclic", [((64,), False), ((16, 24, 24), False), ((24, 20, 20), True)], ids=str)
def test_equal_positions_are_the_plain_rotation(torch, inter, tokens, sections, cyclic):
    """Text tokens, whose positions are the same on every axis, get pa_qk_norm_rope's bits."""
    rng = np.random.default_rng(tokens)
    x, w = up(torch, rows(rng, tokens, 40, 128)), up(torch, (1 + 0.2 * rng.normal(size=128)).astype(np.float16))
    cs, pos = up(torch, table(rng, 90, 128)), up(torch, rng.integers(0, 90, tokens).astype(np.int32))
    outs = []
    for kw in (dict(positions=pos), dict(positions=pos.repeat(len(sections), 1), sections=sections, cyclic=cyclic)):
        qo, ko = (torch.empty((tokens, n, 128), dtype=torch.float16, device="cuda") for n in (32, 8))
        pa.pa_qk_norm_rope(x[:, :32], x[:, 32:], w, w, cs, q_out=qo, k_out=ko, interleaved=inter, **kw)
        outs.append((qo, ko))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_bad_positions_leave_their_token_out(torch):
    rng = np.random.default_rng(5)
    q, k = rows(rng, 6, 4, 64), rows(rng, 6, 2, 64)
    cs = table(rng, 10, 64)
    pos = np.array([[0, 9, 3, -2, -1, 3], [0, 0, 10, 1, 4, 1 << 30], [1, 2, 3, 4, 5, 6]], np.int32)
    dq, dk = up(torch, q), up(torch, k)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = dict(status=status, sections=(10, 11, 11))
    pa.pa_qk_norm_rope(dq, dk, None, None, up(torch, cs), up(torch, pos), dq, dk, **kw)
    assert status.item() == pa.PA_STATUS_BIT_POSITION
    live = ((pos >= 0) & (pos < 10)).all(0)
    assert live.tolist() == [True, True, False, False, False, False]
    for got, part in ((dq, q), (dk, k)):
        got = got.cpu().numpy()
        want, mag = wref.rotate_axes(part[live], None, cs, pos[:, live], (10, 11, 11), False, 0, False)
        check_half(got[live], want, ref.rotate_error(mag, 64))
        np.testing.assert_array_equal(got[~live], part[~live])
    status.zero_()
    pos[:, 2:] = -1  # padding is no error
    pa.pa_qk_norm_rope(dq, dk, None, None, up(torch, cs), up(torch, pos), dq, dk, **kw)
    assert status.item() == 0


# q, ctx, H, Hk, hk, hv, rotary dim, sections, cyclic, interleaved, norm
STORE = [
    ([1, 1], [1, 40], 32, 8, 128, 128, 128, (16, 24, 24), False, False, True),
    ([5, 0, 9], [5, 7, 90], 4, 2, 64, 64, 32, (6, 5, 5), True, True, True),
    ([64], [64], 28, 4, 128, 64, 128, (24, 20, 20), True, False, True),
    ([3, 2], [17, 2], 2, 1, 576, 512, 64, (8, 8, 8, 8), False, True, False),
    ([150, 170], [150, 333], 32, 8, 128, 128, 128, (16, 24, 24), False, False, True),
]


@pytest.mark.parametrize("case", STORE, ids=str)
def test_store(torch, case):
    q, ctx, H, Hk, hk, hv, rot, sections, cyclic, inter, norm = case
    rng = np.random.default_rng(hk + H)
    batch = ref.make_batch(rng, q, ctx, 16)
    T = int(batch.q.sum())
    xq, xk, v = rows(rng, T, H, hk), rows(rng, T, Hk, hk), rows(rng, T, Hk, hv)
    w = [(1 + 0.2 * rng.normal(size=hk)).astype(np.float16) if norm else None for _ in range(2)]
    cs, pos = table(rng, 128, rot), rng.integers(0, 128, (len(sections), T)).astype(np.int32)
    c = empty_cache(torch, batch.num_blocks, 16, Hk, hk, hv)
    qo = torch.zeros((T, H, hk), dtype=torch.float16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.store(up(torch, xq), up(torch, xk), up(torch, v), up(torch, w[0]), up(torch, w[1]), up(torch, cs), up(torch, pos),
            up(torch, batch.tables), up(torch, batch.ctx), up(torch, batch.q), max(q), qo, eps=1e-5, interleaved=inter,
            status=status, sections=sections, cyclic=cyclic)
    assert status.item() == 0
    eps = np.float64(np.float32(1e-5))
    want, mag = wref.rotate_axes(xq, w[0], cs, pos, sections, cyclic, eps, inter)
    check_half(qo.cpu().numpy(), want, ref.rotate_error(mag, hk))
    want_v, want_ve = expected_cache(batch, v, hv, Hk)
    assert ref.same_codes(c.value.view(torch.uint8).cpu().numpy(), want_v)
    np.testing.assert_array_equal(c.value_exps.cpu().numpy(), want_ve)
    # keys: the exponent that a maximum within its fp32 error needs, and every element within half
    # a step of e4m3 and that error
    want, mag = wref.rotate_axes(xk, w[1], cs, pos, sections, cyclic, eps, inter)
    error = 1.001 * ref.rotate_error(mag, hk)
    codes, exps = c.key.view(torch.uint8).cpu().numpy(), c.key_exps.cpu().numpy()
    for b in range(len(q)):
        n, L, t0 = q[b], ctx[b], int(batch.starts[b])
        blk, off = batch.slots(b, L - n, L)
        e = exps[blk, :, off].astype(np.int64) - 127
        y, err = want[t0:t0 + n], error[t0:t0 + n]
        least, most = ref.row_exponent(np.maximum(np.abs(y) - err, 0)), ref.row_exponent(np.abs(y) + err)
        assert ((e >= least) & (e <= most)).all()
        held = ref.decode(codes[blk, off]) * 2.0 ** e[..., None]
        half_step = np.maximum(2.0**-4 * (np.abs(y) + err), 2.0**-10 * 2.0 ** e[..., None])
        assert (np.abs(held - y) <= half_step + err).all()


def test_store_leaves_out_padding_and_bad_positions(torch):
    rng = np.random.default_rng(3)
    batch = ref.make_batch(rng, [4], [20], 16)
    x = rows(rng, 6, 8, 64)
    c = empty_cache(torch, batch.num_blocks, 16, 2, 64, 64)
    before = [t.view(torch.uint8).clone() for t in (c.key, c.value, c.key_exps, c.value_exps)]
    pos = np.array([[3, 3, -1, 3, 0, 0], [3, 11, 3, 3, 0, 0]], np.int32)
    qo = torch.full((6, 4, 64), 7.0, dtype=torch.float16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d = up(torch, x)
    c.store(d[:, :4], d[:, 4:6], d[:, 6:], None, None, up(torch, table(rng, 10, 64)), up(torch, pos),
            up(torch, batch.tables), up(torch, batch.ctx), up(torch, batch.q), 4, qo, status=status, sections=(16, 16))
    assert status.item() == pa.PA_STATUS_BIT_POSITION
    assert (qo[[1, 2, 4, 5]] == 7).all() and not (qo[[0, 3]] == 7).all(-1).any()
    stored = np.zeros((batch.num_blocks, 16), bool)
    blk, off = batch.slots(0, 16, 20)
    stored[blk[[0, 3]], off[[0, 3]]] = True
    keep = ~up(torch, stored)
    for t, old in zip((c.key, c.value), before):
        assert torch.equal(t.view(torch.uint8)[keep], old[keep])
    for t, old in zip((c.key_exps, c.value_exps), before[2:]):
        assert torch.equal(t.transpose(1, 2)[keep], old.transpose(1, 2)[keep])
        assert not bool((t.transpose(1, 2)[~keep] == old.transpose(1, 2)[~keep]).all())


def test_captured_and_replayed_on_another_stream(torch):
    """The captured call takes new positions; so does a call on another stream than the current one."""
    rng = np.random.default_rng(8)
    x, cs = up(torch, rows(rng, 50, 10, 128)), up(torch, table(rng, 60, 128))
    pos = up(torch, rng.integers(0, 60, (3, 50)).astype(np.int32))
    qo, ko = (torch.empty((50, n, 128), dtype=torch.float16, device="cuda") for n in (8, 2))

    def run(stream=None):
        pa.pa_qk_norm_rope(x[:, :8], x[:, 8:], None, None, cs, pos, qo, ko, sections=(16, 24, 24), stream=stream)
    run()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        run()
    for _ in range(2):
        pos.copy_(up(torch, rng.integers(0, 60, (3, 50)).astype(np.int32)))
        qo.zero_()
        g.replay()
        got = qo.clone()
        qo.zero_()
        torch.cuda.synchronize()
        run(s)
        s.synchronize()
        assert torch.equal(got, qo) and bool((got != 0).any())
