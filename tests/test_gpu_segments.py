"""Contexts of which a worker has more than 65536 keys of one row tile: it takes them in segments, whose results
it adds up itself."""
import numpy as np
import pytest

import paged_kv_cache_206_gb300 as pa
from . import window_ref as wref
from .test_gpu_tree import Case as TreeCase
from .test_gpu_window import Case as WindowCase

pytestmark = pytest.mark.gpu

ALL = 2**31 - 1


@pytest.fixture(scope="module")
def torch():
    import torch
    torch.cuda.set_device(0)
    return torch


@pytest.mark.parametrize("value", [1 + 2.0**-7, 1.7001953125])
@pytest.mark.parametrize("call", ["window", "tree"])
@pytest.mark.parametrize("group,q,d", [(1, 1, 64), (2, 1, 128), (2, 1, 256), (8, 2, 128), (8, 10, 128), (8, 10, 64),
                                       (8, 32, 128), (8, 32, 64)])
def test_equal_values_over_a_million_keys(torch, group, q, d, call, value):
    """One SM has it all. An addition of 16 keys to an fp32 sum cuts off less than a step of 2^-23 of the sum, which
    grows evenly over the 4096 of a segment: less than 2^-12 together. Half a step of the result besides (2^-11
    from 1 to 2)."""
    keys, bs, Hk = 2**20, 128, 8
    key = torch.zeros((1, bs, Hk, d), dtype=torch.float16, device="cuda")
    tables = torch.zeros((1, keys // bs), dtype=torch.int32, device="cuda")
    query = torch.ones((q, Hk * group, d), dtype=torch.float16, device="cuda")
    out = torch.full_like(query, 7.0)
    lens, qs = (torch.tensor([n], dtype=torch.int32, device="cuda") for n in (keys, q))
    shape = dict(batch=1, num_heads=Hk * group, max_seqlen_q=q, max_blocks_per_seq=keys // bs)
    args = query, tables, lens, qs
    if call == "window":
        step = pa.WindowStep(key, torch.full_like(key, value), **shape, window=ALL)
    else:
        step, args = pa.TreeStep(key, torch.full_like(key, value), **shape), (*args, None)
    step.cfg.num_sms = 1
    step.run(*args, out)
    assert step.status() == (pa.PA_OK, 0)
    assert (out.double() - value).abs().max().item() <= 2.0**-11 + value * (2.0**-12 + 2.0**-18)


def waves(c, x):
    """Values whose mean moves with the position by more than their spread, so that no part of the keys can
    be left out or weighed wrongly unseen."""
    if not c.real:
        return
    for b, L in enumerate(c.batch.ctx):
        blk, off = c.batch.slots(b, 0, int(L))
        x[blk, off] = x[blk, off] / 8 + (3 * np.sin(np.arange(L) / 17000.0 + b))[:, None, None].astype(np.float16)


# q, ctx, H, Hk, dims, window, sinks, SMs
WINDOWS = [
    ([1], [150000], 8, 4, 128, ALL, 0, 1),
    ([3], [140000], 8, 4, 64, 110000, 20000, 1),
    ([4], [72000], 16, 4, 256, ALL, 0, 1),
    ([1, 2], [80001, 75000], 4, 2, 256, ALL, 0, 1),
    ([20, 1], [150000, 300], 4, 1, 128, ALL, 0, 1),
    ([20], [200000], 4, 1, 64, 150000, 5, 2),
    ([13, 7, 9], [131072, 70000, 65537], 4, 1, 128, ALL, 0, 3),
    ([70], [140001], 2, 1, 128, ALL, 0, 1),
    ([70, 2], [150001, 70000], 4, 1, 128, 60000, 46000, 1),
    ([70, 66], [140001, 70000], 2, 1, 128, 100000, 0, 2),
    ([140], [75000], 2, 1, 64, ALL, 0, 1),
    ([66], [66000], 4, 1, 64, ALL, 66, 1),
]


@pytest.mark.parametrize("case", WINDOWS, ids=str)
@pytest.mark.parametrize("bits", [8, 16])
def test_windows(torch, bits, case):
    q, ctx, H, Hk, d, window, sinks, sms = case
    c = WindowCase(torch, bits, q, ctx, H, Hk, d, d, 128, window, sinks, poison=waves)
    c.step.cfg.num_sms = sms
    first = c.run().clone()
    assert c.step.status() == (pa.PA_OK, 0)
    c.check()
    assert torch.equal(c.run(), first)


# q, ctx, H, Hk, dims, kind, SMs
TREES = [
    ([1], [150000], 8, 4, 128, "chain", 1),
    ([4], [72000], 16, 4, 256, "tree", 1),
    ([16, 3], [100000, 70000], 2, 1, 128, "tree", 1),
    ([16], [150000], 4, 1, 64, "tree", 2),
    ([70], [140000], 2, 1, 128, "tree", 1),
    ([80, 70], [75000, 66000], 4, 1, 64, "tree", 3),
]


@pytest.mark.parametrize("case", TREES, ids=str)
@pytest.mark.parametrize("bits", [8, 16])
def test_trees(torch, bits, case):
    q, ctx, H, Hk, d, kind, sms = case
    c = TreeCase(torch, bits, q, ctx, H, Hk, d, d, 128, kind, poison=waves)
    c.step.cfg.num_sms = sms
    first = c.run().clone()
    assert c.step.status() == (pa.PA_OK, 0)
    c.check()
    assert torch.equal(c.run(), first)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("kind", ["chain", "tree"])
def test_segments_without_keys(torch, bits, kind):
    """The last segment begins behind the own last key of the first row tile, of 64 tokens."""
    c = TreeCase(torch, bits, [66, 3], [65538, 90], 4, 1, 64, 64, 128, kind, poison=waves)
    c.step.cfg.num_sms = 1
    c.run()
    assert c.step.status() == (pa.PA_OK, 0)
    c.check()


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("q,H,d", [(2, 4, 128), (20, 4, 128), (70, 4, 128), (70, 4, 64)])
def test_values_that_are_no_numbers_stay_in_the_rows_that_see_them(torch, bits, q, H, d):
    """One at the start of a window that the first rows see, in a segment before the last one; one that all see in
    another; one among the current tokens."""
    ctx, window = 290000 + q, 200000
    first = ctx - q - window + 1  # the first row's first key
    places = [(first + q // 2, 2), (first + 100000, 5), (ctx - q // 2 - 1, 9)]

    def poison(c, x):
        if c.real:
            for at, dim in places:
                blk, off = c.batch.slots(0, at, at + 1)
                x[blk[0], off[0], 0, dim] = np.nan

    c = WindowCase(torch, bits, [q], [ctx], H, 1, d, d, 128, window, 0, poison=poison)
    c.step.cfg.num_sms = 1
    got = c.run().cpu().numpy()
    assert c.step.status() == (pa.PA_OK, 0)
    see = wref.sees(q, ctx, window, 0)
    for at, dim in places:
        assert (np.isnan(got[..., dim]) == see[:, at][:, None]).all(), at
    others = np.delete(got, [dim for _, dim in places], axis=2)
    assert np.isfinite(others).all()
    want, bound = c.want()
    assert (np.abs(others - np.delete(want, [dim for _, dim in places], axis=2))
            <= np.delete(bound, [dim for _, dim in places], axis=2)).all()


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("q,H,Hk,d", [(1, 8, 2, 128), (4, 8, 2, 64), (3, 16, 4, 256), (16, 8, 2, 128), (40, 8, 2, 64),
                                      (200, 4, 1, 128), (2, 6, 2, 96)])
def test_the_forms_with_segments_give_the_same_bits(torch, bits, q, H, Hk, d):
    """A batch of short contexts under tables that allow long ones."""
    qs = [q, 1, q, max(q // 2, 1)] * 9
    ctx = [n + 37 * i + 5 for i, n in enumerate(qs)]
    window = WindowCase(torch, bits, qs, ctx, H, Hk, d, d, 64, 70000, 20)
    tree = TreeCase(torch, bits, qs, ctx, H, Hk, d, d, 64, "tree")
    for c, call, more in ((window, pa.WindowStep, dict(window=70000, sinks=20)), (tree, pa.TreeStep, {})):
        want = c.run().clone()
        wide = torch.full((len(qs), 2048), -1, dtype=torch.int32, device="cuda")
        wide[:, :c.args[1].shape[1]] = c.args[1]
        (k, ke), (v, ve) = c.dev
        step = call(k, v, ke, ve, batch=len(qs), num_heads=H, max_seqlen_q=max(qs), max_blocks_per_seq=2048, **more)
        out = torch.full_like(c.out, 7.0)
        step.run(c.args[0], wide, *c.args[2:], out)
        assert step.status() == c.step.status() == (pa.PA_OK, 0)
        assert torch.equal(out, want)


def test_the_workspace_of_long_contexts_has_room_for_them(torch):
    """A third slot a worker where a tile may have more than 65536 keys, and only there."""
    def need(keys, **kw):
        cfg = pa.make_config(batch=2, num_heads=32, kv_heads=8, head_size_k=128, head_size_v=128, block_size=128,
                             num_blocks=16, max_blocks_per_seq=keys // 128, max_seqlen_q=kw.pop("q"),
                             mask_type=pa.PA_MASK_NONE, num_sms=152)
        return pa.pa_window_workspace(cfg, pa.pa_window(**kw)) if kw else pa.pa_tree_workspace(cfg)
    for q in (1, 16, 100):
        assert need(65536, q=q) == need(128, q=q) < need(65536 + 128, q=q) < 2 * need(128, q=q)
        assert need(2**30, q=q, window=65000, sinks=280) == need(128, q=q, window=1, sinks=0)
        assert need(2**30, q=q, window=65000, sinks=537) == need(2**30, q=q, window=ALL, sinks=0) == need(2**30, q=q)


@pytest.mark.parametrize("bits", [8, 16])
@pytest.mark.parametrize("q,d", [(1, 128), (4, 256), (16, 128), (16, 64), (300, 128)])
def test_waits_that_run_out_in_the_kernels_that_take_segments(torch, bits, q, d):
    """Tables that allow long tiles, under a limit of a few cycles: PA_ERR_TIMEOUT, and with the default limit
    the same bits as before."""
    g = torch.Generator(device="cuda").manual_seed(q)
    B, H, Hk, bs, cols = 24, 32, 8, 64, 2048
    lens = torch.randint(q, 6000, (B,), generator=g, device="cuda", dtype=torch.int32)
    qs = torch.full_like(lens, q)
    tables = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
    blocks = B * 94
    tables[:, :94] = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32).view(B, 94)
    k, v = (torch.randn((blocks, bs, Hk, d), generator=g, device="cuda").half() for _ in range(2))
    exps = [None, None]
    if bits == 8:
        k, v = k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn)
        exps = [torch.randint(125, 129, (blocks, Hk, bs), generator=g, device="cuda").to(torch.uint8) for _ in range(2)]
    query = torch.randn((B * q, H, d), generator=g, device="cuda").half()
    flush = torch.empty(512 << 20, dtype=torch.uint8, device="cuda")
    shape = dict(batch=B, num_heads=H, max_seqlen_q=q, max_blocks_per_seq=cols)
    for step in (pa.WindowStep(k, v, *exps, **shape, window=ALL), pa.TreeStep(k, v, *exps, **shape)):
        out = torch.empty_like(query)
        args = (query, tables, lens, qs, out) if isinstance(step, pa.WindowStep) else (query, tables, lens, qs, None, out)
        first = step.run(*args).clone()
        assert step.status() == (pa.PA_OK, 0)
        for _ in range(10):  # whether a wait outlasts 32 cycles depends on when its copy lands
            flush.zero_()
            pa.testing_set_wait_limit(32)
            try:
                step.run(*args)
                st, word = step.status()
            finally:
                pa.testing_set_wait_limit(0)
            if st == pa.PA_ERR_TIMEOUT:
                break
        assert (st, word) == (pa.PA_ERR_TIMEOUT, pa.PA_STATUS_BIT_TIMEOUT)
        pa.pa_status_clear(step.workspace)
        step.run(*args)
        assert step.status() == (pa.PA_OK, 0)
        assert torch.equal(out, first)
