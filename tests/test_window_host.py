"""Host side of pa_window.h, pa_blocks.h and the calls with positions of several axes, without a
GPU: the references against other statements of the same, and every refusal."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_206_gb300 as pa
from paged_kv_cache_206_gb300 import build_lib
from . import serving_ref as ref
from . import window_ref as wref

FAKE, OTHER = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21)
BAD = ctypes.c_void_p((1 << 20) + 8)
INVALID = pa.PA_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return pa.load_library()


# ---- the references

def test_a_wide_window_is_the_causal_chain():
    rng = np.random.default_rng(0)
    batch = ref.make_batch(rng, [3, 0, 5], [20, 7, 5], 16)
    q = rng.normal(size=(8, 4, 16))
    k, v = (rng.normal(size=(batch.num_blocks, 16, 2, 16)) for _ in range(2))
    ev = np.zeros((batch.num_blocks, 2, 16))
    for window, sinks in ((20, 0), (10**9, 3), (1, 20)):
        got = wref.window_attention(q, k, v, ev, batch, window, sinks, 0.25)
        want = ref.tree_attention(q, k, v, ev, ev, batch, None, 0.25)
        for a, b in zip(got, want):
            np.testing.assert_allclose(a, b, rtol=1e-12)


def test_which_keys_a_token_attends():
    see = wref.sees(2, 7, 3, 1)
    assert see.astype(int).tolist() == [[1, 0, 0, 1, 1, 1, 0], [1, 0, 0, 0, 1, 1, 1]]


def test_one_axis_is_the_plain_rotation():
    rng = np.random.default_rng(1)
    x, cs = rng.normal(size=(5, 3, 64)), rng.normal(size=(9, 32))
    pos = rng.integers(0, 9, 5)
    for cyclic, sections in ((False, (16,)), (True, (16,)), (False, (4, 0, 12)), (True, (6, 5, 5))):
        got = wref.rotate_axes(x, None, cs, np.stack([pos] * len(sections)), sections, cyclic, 0, False)
        for a, b in zip(got, ref.rotate(x, None, cs, pos, 0, False)):
            np.testing.assert_allclose(a, b, rtol=1e-12)
    assert wref.axis_of_pair((2, 1, 3), False, 6) == [0, 0, 1, 2, 2, 2]
    assert wref.axis_of_pair((4, 2, 1), True, 7) == [0, 1, 2, 0, 1, 0, 0]


def test_what_is_taken_and_given_back_leaves_the_pool_as_it_was():
    p = wref.Pool(3, 8, 20, 16)
    slots, positions, _ = p.step([70, 16, 41], [65, 0, 1], 67)
    assert p.held == [5, 1, 3] and p.tables[1][0] == 5 and p.count == 11
    assert slots[64:] == [4 * 16 + 5, 8 * 16 + 8, -1] and positions[:2] + positions[64:] == [5, 6, 69, 40, -1]
    p.step([0, 0, 0], [0, 0, 0], 0)
    assert p.free == list(range(19, -1, -1)) and p.count == 20 and p.held == [0, 0, 0]


# ---- refusals of the library

def cfg(**kw):
    base = dict(batch=2, num_heads=8, kv_heads=2, head_size_k=64, block_size=16, num_blocks=4,
                max_blocks_per_seq=2, max_seqlen_q=4, num_sms=4)
    base.update(kw)
    return pa.make_config(**base)


def test_window_refusals(lib):
    win = pa.pa_window(4, 1)
    need = pa.pa_window_workspace(cfg(), win)

    def call(c=None, w=win, **kw):
        a = dict(tokens=0, q=FAKE, kc=FAKE, vc=OTHER, ke=None, ve=None, bt=FAKE, cl=FAKE, ql=FAKE, ws=FAKE,
                 n=1 << 30, out=OTHER)
        a.update(kw)
        return lib.pa_window_forward(ctypes.byref(cfg() if c is None else c), None if w is None else ctypes.byref(w),
                                     a["tokens"], a["q"], a["kc"], a["vc"], a["ke"], a["ve"], a["bt"], a["cl"],
                                     a["ql"], a["ws"], a["n"], a["out"], None)
    assert call() == pa.PA_OK and call(ql=None) == pa.PA_OK
    assert call(ke=FAKE, ve=OTHER) == pa.PA_OK
    assert call(n=need) == pa.PA_OK
    assert call(n=need - 1) == pa.PA_ERR_BUFFER_TOO_SMALL
    for kw in (dict(tokens=-1), dict(q=None), dict(kc=None), dict(vc=None), dict(vc=FAKE), dict(ke=FAKE),
               dict(ve=FAKE), dict(ke=FAKE, ve=FAKE), dict(bt=None), dict(cl=None), dict(ws=None),
               dict(out=None), dict(q=BAD), dict(kc=BAD), dict(vc=BAD), dict(ke=BAD, ve=OTHER),
               dict(out=BAD), dict(ws=ctypes.c_void_p((1 << 20) + 16)), dict(w=None),
               dict(w=pa.pa_window(0, 0)), dict(w=pa.pa_window(-1, 0)), dict(w=pa.pa_window(1, -1))):
        assert call(**kw) == INVALID, kw
    assert call(w=pa.pa_window(2**31 - 1, 2**31 - 1)) == pa.PA_OK
    for kw in (dict(mask_type=1), dict(mask_type=2), dict(mask_type=5), dict(chunk_blocks=2),
               dict(num_sms=0), dict(num_sms=65536), dict(num_heads=7), dict(head_size_k=24),
               dict(block_size=144), dict(batch=0), dict(max_blocks_per_seq=0)):
        assert call(cfg(**kw)) == INVALID, kw
    assert call(cfg(mask_type=4)) == pa.PA_ERR_UNSUPPORTED
    assert call(tokens=1, out=FAKE) == INVALID  # the query as output
    assert lib.pa_window_workspace(ctypes.byref(cfg()), ctypes.byref(win), None) == INVALID
    for tokens in (2**31, 2**58, 2**60, 2**61, 2**62, 2**63 - 1):
        for d in (64, 128, 272):
            assert call(cfg(head_size_k=d), tokens=tokens, n=1 << 40) == INVALID


BLOCKS = dict(batch=2, block_size=16, num_blocks=4, max_blocks_per_seq=2, window=0, sinks=0)


def test_blocks_refusals(lib):
    P = [ctypes.c_void_p((2 + n) << 20) for n in range(9)]

    def call(c=None, **kw):
        a = dict(cl=P[0], ql=P[1], bt=P[2], held=P[3], gone=P[4], free=P[5], count=P[6], tokens=-1, slots=P[7],
                 pos=P[8])
        a.update(kw)
        return lib.pa_blocks_step(ctypes.byref(pa.pa_blocks_config(**{**BLOCKS, **(c or {})})), a["cl"], a["ql"],
                                  a["bt"], a["held"], a["gone"], a["free"], a["count"], a["tokens"], a["slots"],
                                  a["pos"], None, None)
    # (every call is one that is refused: a good one would launch)
    assert call() == INVALID
    for kw in (dict(cl=None), dict(bt=None), dict(held=None), dict(gone=None), dict(free=None), dict(count=None),
               dict(held=P[4]), dict(count=P[3]), dict(free=P[3]), dict(bt=P[5]), dict(tokens=2**30),
               dict(tokens=2**62), dict(slots=ctypes.c_void_p((9 << 20) + 4)), dict(pos=ctypes.c_void_p((9 << 20) + 2)),
               dict(cl=ctypes.c_void_p((2 << 20) + 1)), dict(count=ctypes.c_void_p((8 << 20) + 3))):
        assert call(**{"tokens": 0, **kw}) == INVALID, kw
    for c in (dict(batch=0), dict(batch=2049), dict(block_size=0), dict(block_size=24), dict(num_blocks=0),
              dict(max_blocks_per_seq=0), dict(window=-1), dict(sinks=-1), dict(num_blocks=1 << 27),
              dict(batch=2048, max_blocks_per_seq=1 << 20)):
        assert call(c, tokens=0) == INVALID, c


ROT = dict(num_heads=4, kv_heads=2, head_size=64, rotary_dim=64, interleaved=0, max_positions=8, eps=1e-6)
CACHE = dict(batch=2, kv_heads=2, head_size_k=64, head_size_v=64, block_size=16, num_blocks=4,
             max_blocks_per_seq=2, max_rows=1)
GOOD_AXES = [(1, 0, (32,)), (1, 1, (32,)), (3, 0, (8, 12, 12)), (3, 0, (32, 0, 0)), (3, 0, (0, 0, 32)),
             (3, 1, (11, 11, 10)), (3, 1, (12, 10, 10)), (4, 1, (8, 8, 8, 8)), (2, 1, (32, 0))]
BAD_AXES = [(0, 0, ()), (5, 0, (8, 8, 8, 8)), (-1, 0, (32,)), (3, 0, (8, 12, 11)), (3, 0, (8, 12, 13)),
            (3, 0, (-4, 18, 18)), (3, 1, (10, 11, 11)), (2, 1, (15, 17)), (4, 1, (5, 9, 9, 9))]


def axes(count, cyclic, sections):
    return pa.pa_axes(count, cyclic, (ctypes.c_int32 * 4)(*sections))


def test_axes_refusals(lib):
    def rotate(a, pos=FAKE, tokens=0):
        return lib.pa_qk_norm_rope_axes(ctypes.byref(pa.pa_rotary(**ROT)), None if a is None else ctypes.byref(a),
                                        tokens, FAKE, 256, FAKE, 128, FAKE, FAKE, FAKE, pos, FAKE, OTHER, None, None)

    def store(a, pos=FAKE, tokens=0):
        return lib.pa_cache_store_axes(ctypes.byref(pa.pa_cache_config(**CACHE)), ctypes.byref(pa.pa_rotary(**ROT)),
                                       None if a is None else ctypes.byref(a), tokens, FAKE, 256, FAKE, 128, FAKE,
                                       128, None, None, FAKE, pos, FAKE, FAKE, None, FAKE, FAKE, OTHER, OTHER, OTHER,
                                       None, None)
    for call in (rotate, store):
        for a in GOOD_AXES:
            assert call(axes(*a)) == pa.PA_OK, a
        for a in BAD_AXES:
            assert call(axes(*a)) == INVALID, a
        assert call(None) == INVALID
        assert call(axes(*GOOD_AXES[2]), pos=None) == INVALID
        for tokens in (-1, 2**31, 2**60, 2**63 - 1):
            assert call(axes(*GOOD_AXES[2]), tokens=tokens) == INVALID


# ---- refusals of the binding

def refused(f, *a, **kw):
    with pytest.raises(pa.PaError) as e:
        f(*a, **kw)
    assert e.value.status == INVALID
    return str(e.value)


def test_binding_refuses_what_the_library_cannot_see(lib):
    f16 = torch.float16
    k = torch.zeros((3, 16, 2, 64), dtype=f16)
    step = dict(batch=2, num_heads=4, max_seqlen_q=1, max_blocks_per_seq=2)
    assert "CUDA" in refused(pa.WindowStep, k, k.clone(), **step, window=4)
    for kw in (dict(window=0), dict(window=-3), dict(window=2**31), dict(window=4, sinks=-1)):
        assert "window" in refused(pa.WindowStep, k, k.clone(), **step, **kw)

    pool = pa.BlockPool.empty(2, 4, 6, 16, device="cpu")
    lens = torch.ones(2, dtype=torch.int32)
    assert "CUDA" in refused(pool.step, lens)
    slots, pos = torch.zeros(5, dtype=torch.int64), torch.zeros(5, dtype=torch.int32)
    assert "CUDA" in refused(pool.step, lens, lens, slots, pos)
    for a in ((lens.long(),), (lens[:1],), (lens, lens.long()), (lens, lens, pos), (lens, lens, slots, slots),
              (lens, lens, slots, pos[:4]), (lens, lens, slots[::2], None), (lens, lens, slots.view(5, 1), None)):
        assert "CUDA device" not in refused(pool.step, *a)
    parts = dict(block_tables=pool.block_tables, held=pool.held, gone=pool.gone, free=pool.free, count=pool.count,
                 block_size=16)
    for kw in (dict(block_tables=pool.block_tables.long()), dict(block_tables=pool.held), dict(held=pool.held[:1]),
               dict(gone=pool.gone.long()), dict(free=pool.block_tables), dict(count=pool.held), dict(window=-1),
               dict(sinks=-1), dict(block_size=-16)):
        refused(pa.BlockPool, **{**parts, **kw})

    q, table = torch.zeros((5, 4, 64), dtype=f16), torch.zeros((9, 32))
    kk, pos = torch.zeros((5, 2, 64), dtype=f16), torch.zeros((3, 5), dtype=torch.int32)
    args = dict(query=q, key=kk, q_weight=None, k_weight=None, cos_sin=table, positions=pos, q_out=q.clone(),
                k_out=kk.clone(), sections=(4, 6, 6))
    assert "CUDA" in refused(pa.pa_qk_norm_rope, **args)
    for kw in (dict(positions=None), dict(positions=pos[0]), dict(positions=pos[:2]), dict(positions=pos.t()),
               dict(sections=(4, 12)), dict(sections=()), dict(sections=(4, 4, 4, 2, 2)), dict(sections=None),
               dict(sections=(4, -6, 18))):
        assert "CUDA device" not in refused(pa.pa_qk_norm_rope, **{**args, **kw})
    cache = pa.QuantCache.empty(3, 16, 2, 64, device="cpu")
    lens = torch.ones(5, dtype=torch.int32)
    tables = torch.zeros((5, 1), dtype=torch.int32)
    args = (q, kk, kk, None, None, table)
    rest = (tables, lens, None, 1, q.clone())
    assert "CUDA" in refused(cache.store, *args, pos, *rest, sections=(4, 6, 6))
    assert "CUDA device" not in refused(cache.store, *args, None, *rest, sections=(4, 6, 6))
    assert "CUDA device" not in refused(cache.store, *args, pos[0], *rest, sections=(4, 6, 6))


def test_an_axes_configuration_lives_as_long_as_its_call(monkeypatch, lib):
    import weakref

    from paged_kv_cache_206_gb300 import serving
    rows, ints = torch.zeros((1, 2, 64), dtype=torch.float16), torch.ones((2, 1), dtype=torch.int32)
    serving._axes.clear()
    seen = []

    def launch(where, at, stream, function, *args):
        used = [weakref.ref(c) for a, c in serving._axes.values() if a in args]
        serving._axes.clear()
        seen.append(len(used))
        assert all(c() is not None for c in used)

    monkeypatch.setattr(serving, "_launch", launch)
    table = torch.zeros((2, 64))
    pa.pa_qk_norm_rope(rows, rows, None, None, table, ints, rows.clone(), rows.clone(), sections=(16, 16))
    assert seen == [1]


@pytest.mark.parametrize("module", [True, False])
def test_calls_of_13_and_24_arguments(monkeypatch, lib, module):
    """With the C module and without it every argument comes to its place (the last but one wrong: refused)."""
    from paged_kv_cache_206_gb300 import serving
    monkeypatch.setattr(serving, "_f16", None)
    if not module:
        monkeypatch.setattr(build_lib, "CALL", "/nonexistent")
    serving._start()
    a, c, r = axes(*GOOD_AXES[2]), pa.pa_cache_config(**CACHE), pa.pa_rotary(**ROT)
    F, O = FAKE.value, OTHER.value

    def store(q_out, tokens=0):
        return serving._call(serving._store_axes, ctypes.addressof(c), ctypes.addressof(r), ctypes.addressof(a), tokens,
                             F, 256, F, 128, F, 128, None, None, F, F, F, F, None, F, F, O, O, q_out, None, 0)
    assert store(O) == pa.PA_OK
    assert store(O + 8) == INVALID and store(None) == INVALID and store(O, -1) == INVALID
    b = pa.pa_blocks_config(**BLOCKS)
    pool = F + 256, F + 512, F + 768, F + 1024, F + 1280
    assert serving._call(serving._blocks, ctypes.addressof(b), F, F, *pool, -1, F, F, None, 0) == INVALID
    monkeypatch.undo()
    serving._start()
