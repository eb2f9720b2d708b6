"""Host side of pa_cache.h and pa_tree.h, without a GPU: the reference's own
8-bit element against torch's, and every refusal."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_206_gb300 as pa
from paged_kv_cache_206_gb300 import build_lib
from . import serving_ref as ref

FAKE = ctypes.c_void_p(1 << 20)
OTHER = ctypes.c_void_p(1 << 21)
BAD = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return pa.load_library()


def test_reference_codes_are_torchs():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref.decode(codes), want)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(size=4000) * 2.0 ** rng.integers(-12, 9, 4000), want[:127],
                        (want[:126] + want[1:127]) / 2, [0.0, -0.0, 448.0, 464.0]])
    x = x[np.abs(x) <= 448]
    got = torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(ref.encode(x.astype(np.float32).astype(np.float64)), got)


def test_reference_exponent_at_its_borders():
    x = np.array([[448.0, 1], [449, 1], [0, 0], [np.inf, 3.5], [np.nan, 3.501], [65504, 0],
                  [2.0**-24, 0]])
    assert ref.row_exponent(x).tolist() == [0, 1, -32, -7, -6, 8, -32]


ROT = dict(num_heads=4, kv_heads=2, head_size=64, rotary_dim=64, interleaved=0, max_positions=8,
           eps=1e-6)


def rotary(**kw):
    return pa.pa_rotary(**{**ROT, **kw})


CACHE = dict(batch=2, kv_heads=2, head_size_k=64, head_size_v=64, block_size=16, num_blocks=4,
             max_blocks_per_seq=2, max_rows=1)


def cache(**kw):
    return pa.pa_cache_config(**{**CACHE, **kw})


def call_rotate(lib, rot=None, **kw):
    a = dict(tokens=0, q=FAKE, qs=256, k=FAKE, ks=128, qw=FAKE, kw=FAKE, cs=FAKE, pos=FAKE, qo=FAKE,
             ko=OTHER)
    a.update(kw)
    return lib.pa_qk_norm_rope(ctypes.byref(rotary() if rot is None else rot), a["tokens"], a["q"],
                               a["qs"], a["k"], a["ks"], a["qw"], a["kw"], a["cs"], a["pos"], a["qo"],
                               a["ko"], None, None)


def test_rotate_refusals(lib):
    assert call_rotate(lib) == pa.PA_OK  # no tokens: nothing to launch
    for kw in (dict(tokens=-1), dict(q=None), dict(k=None), dict(cs=None), dict(pos=None),
               dict(qo=None), dict(ko=None), dict(qo=OTHER), dict(qs=255), dict(qs=248), dict(ks=127),
               dict(qs=260), dict(q=BAD), dict(qw=BAD), dict(cs=BAD), dict(qo=BAD), dict(ko=BAD),
               dict(qs=512), dict(k=OTHER, ks=384)):
        assert call_rotate(lib, **kw) == pa.PA_ERR_INVALID_ARG, kw
    assert call_rotate(lib, qs=512, qo=ctypes.c_void_p(3 << 20)) == pa.PA_OK
    for kw in (dict(num_heads=0), dict(kv_heads=0), dict(head_size=0), dict(head_size=24),
               dict(head_size=592), dict(rotary_dim=-16), dict(rotary_dim=8), dict(rotary_dim=80),
               dict(max_positions=0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        assert call_rotate(lib, rotary(**kw)) == pa.PA_ERR_INVALID_ARG, kw
    assert call_rotate(lib, rotary(rotary_dim=0), cs=None, qw=None, kw=None) == pa.PA_OK


def call_write(lib, cfg=None, store=None, **kw):
    a = dict(tokens=0, q=FAKE, qs=256, k=FAKE, ks=128, v=FAKE, vs=128, bt=FAKE, cl=FAKE, ql=None,
             kc=FAKE, ke=FAKE, vc=OTHER, ve=OTHER, qo=OTHER, cs=FAKE)
    a.update(kw)
    c = ctypes.byref(cache() if cfg is None else cfg)
    if store is None:
        return lib.pa_cache_write(c, a["tokens"], a["k"], a["ks"], a["v"], a["vs"], a["bt"], a["cl"],
                                  a["ql"], a["kc"], a["ke"], a["vc"], a["ve"], None, None)
    return lib.pa_cache_store(c, ctypes.byref(store), a["tokens"], a["q"], a["qs"], a["k"], a["ks"],
                              a["v"], a["vs"], None, None, a["cs"], None, a["bt"], a["cl"], a["ql"],
                              a["kc"], a["ke"], a["vc"], a["ve"], a["qo"], None, None)


def test_write_and_store_refusals(lib):
    for store in (None, rotary()):
        assert call_write(lib, store=store) == pa.PA_OK
        for kw in (dict(tokens=-1), dict(k=None), dict(v=None), dict(bt=None), dict(cl=None),
                   dict(kc=None), dict(ke=None), dict(vc=None), dict(ve=None), dict(vc=FAKE),
                   dict(ve=FAKE), dict(ks=120), dict(vs=129), dict(k=BAD), dict(v=BAD), dict(kc=BAD),
                   dict(ke=BAD), dict(vc=BAD), dict(ve=BAD)):
            assert call_write(lib, store=store, **kw) == pa.PA_ERR_INVALID_ARG, kw
        for kw in (dict(batch=0), dict(batch=2049), dict(kv_heads=0), dict(head_size_k=0),
                   dict(head_size_v=8), dict(head_size_k=592), dict(block_size=8), dict(block_size=0),
                   dict(num_blocks=0), dict(max_blocks_per_seq=0), dict(max_rows=-1),
                   dict(num_blocks=1 << 27, block_size=16)):
            assert call_write(lib, cache(**kw), store=store) == pa.PA_ERR_INVALID_ARG, kw
    assert call_write(lib, store=rotary(kv_heads=4)) == pa.PA_ERR_INVALID_ARG
    assert call_write(lib, store=rotary(head_size=128)) == pa.PA_ERR_INVALID_ARG
    for kw in (dict(q=None), dict(qo=None), dict(qo=BAD), dict(qs=200), dict(cs=None),
               dict(qo=FAKE, qs=512)):
        assert call_write(lib, store=rotary(), **kw) == pa.PA_ERR_INVALID_ARG, kw


def test_read_refusals(lib):
    def call(cfg=None, **kw):
        a = dict(kc=FAKE, ke=FAKE, vc=OTHER, ve=OTHER, bt=FAKE, st=None, cl=FAKE, os=FAKE, rows=0,
                 ko=FAKE, vo=OTHER)
        a.update(kw)
        return lib.pa_cache_read(ctypes.byref(cache() if cfg is None else cfg), a["kc"], a["ke"], a["vc"],
                                 a["ve"], a["bt"], a["st"], a["cl"], a["os"], a["rows"], a["ko"],
                                 a["vo"], None, None)
    assert call() == pa.PA_OK
    assert call(cache(max_rows=0), rows=5) == pa.PA_OK
    for kw in (dict(kc=None), dict(ve=None), dict(bt=None), dict(cl=None), dict(os=None),
               dict(rows=-1), dict(ko=None), dict(vo=None), dict(vo=FAKE), dict(ko=BAD), dict(vo=BAD),
               dict(vc=FAKE)):
        assert call(**kw) == pa.PA_ERR_INVALID_ARG, kw
    assert call(cache(block_size=24)) == pa.PA_ERR_INVALID_ARG


def tree_cfg(**kw):
    base = dict(batch=2, num_heads=8, kv_heads=2, head_size_k=64, block_size=16, num_blocks=4,
                max_blocks_per_seq=2, max_seqlen_q=4, num_sms=4)
    base.update(kw)
    return pa.make_config(**base)


def test_tree_refusals(lib):
    need = pa.pa_tree_workspace(tree_cfg())

    def call(cfg=None, **kw):
        a = dict(tokens=0, q=FAKE, kc=FAKE, vc=OTHER, ke=None, ve=None, bt=FAKE, cl=FAKE, ql=FAKE,
                 par=FAKE, ws=FAKE, n=1 << 30, out=FAKE)
        a.update(kw)
        return lib.pa_tree_forward(ctypes.byref(tree_cfg() if cfg is None else cfg), a["tokens"], a["q"],
                                   a["kc"], a["vc"], a["ke"], a["ve"], a["bt"], a["cl"], a["ql"],
                                   a["par"], a["ws"], a["n"], a["out"], None)
    assert call() == pa.PA_OK
    assert call(ke=FAKE, ve=OTHER) == pa.PA_OK
    assert call(n=need) == pa.PA_OK
    assert call(n=need - 1) == pa.PA_ERR_BUFFER_TOO_SMALL
    for kw in (dict(tokens=-1), dict(q=None), dict(kc=None), dict(vc=None), dict(vc=FAKE), dict(ke=FAKE),
               dict(ve=FAKE), dict(ke=FAKE, ve=FAKE), dict(bt=None), dict(cl=None), dict(ws=None),
               dict(out=None), dict(q=BAD), dict(kc=BAD), dict(vc=BAD), dict(ke=BAD, ve=OTHER),
               dict(out=BAD), dict(ws=ctypes.c_void_p((1 << 20) + 16))):
        assert call(**kw) == pa.PA_ERR_INVALID_ARG, kw
    assert call(tree_cfg(max_seqlen_q=257)) == pa.PA_ERR_INVALID_ARG
    assert call(tree_cfg(max_seqlen_q=257), par=None) == pa.PA_OK
    for kw in (dict(mask_type=1), dict(mask_type=2), dict(mask_type=5), dict(chunk_blocks=2),
               dict(num_sms=0), dict(num_heads=7), dict(head_size_k=24), dict(block_size=144),
               dict(batch=0), dict(max_blocks_per_seq=0)):
        assert call(tree_cfg(**kw)) == pa.PA_ERR_INVALID_ARG, kw
    assert call(tree_cfg(mask_type=4)) == pa.PA_ERR_UNSUPPORTED
    assert lib.pa_tree_workspace(ctypes.byref(tree_cfg()), None) == pa.PA_ERR_INVALID_ARG


def test_binding_refuses_what_the_library_cannot_see():
    f16, e4 = torch.float16, torch.float8_e4m3fn
    nb, bs, hk, d = 3, 16, 2, 64

    def parts(**kw):
        a = dict(key=torch.zeros((nb, bs, hk, d), dtype=e4), value=torch.zeros((nb, bs, hk, d), dtype=e4),
                 key_exps=torch.zeros((nb, hk, bs), dtype=torch.uint8),
                 value_exps=torch.zeros((nb, hk, bs), dtype=torch.uint8))
        a.update(kw)
        return a

    def refused(f, *a, **kw):
        with pytest.raises(pa.PaError) as e:
            f(*a, **kw)
        assert e.value.status == pa.PA_ERR_INVALID_ARG
        return str(e.value)

    c = pa.QuantCache(**parts())
    refused(pa.QuantCache, **parts(key_exps=None))
    refused(pa.QuantCache, **parts(key=torch.zeros((nb, bs, hk, d), dtype=f16)))
    refused(pa.QuantCache, **parts(value=torch.zeros((nb, bs, hk + 1, d), dtype=e4)))
    refused(pa.QuantCache, **parts(key_exps=torch.zeros((nb, bs, hk), dtype=torch.uint8)))
    refused(pa.QuantCache, **parts(value_exps=torch.zeros((nb, hk, bs), dtype=torch.int8)))
    k = torch.zeros((5, hk, d), dtype=f16)
    tables, ones = torch.zeros((5, 2), dtype=torch.int32), torch.ones(5, dtype=torch.int32)
    assert "CUDA" in refused(c.write, k, k, tables, ones)  # everything else is in order
    refused(c.write, k.float(), k, tables, ones)
    refused(c.write, k, k[:4], tables, ones)
    refused(c.write, k, k.transpose(1, 2).contiguous().transpose(1, 2), tables, ones)
    refused(c.write, k, k, tables.long(), ones)
    refused(c.write, k, k, tables, ones[:4])
    refused(c.write, k, k, tables, ones, torch.ones(5, dtype=torch.int64))
    refused(c.write, k, k, tables, ones, status=torch.zeros(1, dtype=torch.int64))
    out = torch.zeros((7, hk, d), dtype=f16)
    assert "CUDA" in refused(c.read, tables, None, ones, ones, 2, out, out.clone())
    refused(c.read, tables, None, ones, ones[:3], 2, out, out.clone())
    refused(c.read, tables, None, ones, ones, 2, out, out[:6])
    refused(c.read, tables, None, ones, ones, 2, out.transpose(0, 1), out)
    q, table = torch.zeros((5, 4, d), dtype=f16), torch.zeros((9, 32))
    args = dict(query=q, key=k, q_weight=None, k_weight=torch.ones(d, dtype=f16), cos_sin=table,
                positions=ones, q_out=q.clone(), k_out=k.clone())
    assert "CUDA" in refused(pa.pa_qk_norm_rope, **args)
    for kw in (dict(k_weight=torch.ones(d)), dict(k_weight=torch.ones(d - 1, dtype=f16)),
               dict(cos_sin=table.double()), dict(cos_sin=table[0]), dict(cos_sin=table[:, :16]),
               dict(positions=None), dict(positions=ones[:4]), dict(positions=ones.long()),
               dict(q_out=q[:4]), dict(k_out=q), dict(key=k[:4]), dict(query=q[0])):
        refused(pa.pa_qk_norm_rope, **{**args, **kw})
    refused(pa.TreeStep, c.key, c.value, batch=5, num_heads=4, max_seqlen_q=1, max_blocks_per_seq=2)


def test_tree_refuses_its_query_as_output_and_too_many_sms(lib):
    def call(cfg, out):
        return lib.pa_tree_forward(ctypes.byref(cfg), 1, FAKE, FAKE, OTHER, None, None, FAKE, FAKE, FAKE,
                                   FAKE, FAKE, 1 << 30, out, None)
    assert call(tree_cfg(), FAKE) == pa.PA_ERR_INVALID_ARG
    assert call(tree_cfg(num_sms=65536), OTHER) == pa.PA_ERR_INVALID_ARG
    need = ctypes.c_size_t()
    assert lib.pa_tree_workspace(ctypes.byref(tree_cfg(num_sms=65535)), ctypes.byref(need)) == pa.PA_OK


def test_tensors_off_the_gpu_are_refused():
    f16 = torch.float16
    cache = pa.QuantCache.empty(2, 16, 2, 64, device="cpu")
    rows, ints = torch.zeros((1, 2, 64), dtype=f16), torch.ones(1, dtype=torch.int32)
    table = torch.zeros((1, 1), dtype=torch.int32)
    out = torch.zeros((1, 2, 64), dtype=f16)
    for call in (lambda: cache.write(rows, rows, table, ints),
                 lambda: cache.store(rows, rows, rows, None, None, None, None, table, ints, None, 1, out),
                 lambda: cache.read(table, None, ints, torch.zeros_like(ints), 1, out, rows),
                 lambda: pa.pa_qk_norm_rope(rows, rows, None, None, None, ints, out, torch.zeros_like(out)),
                 lambda: pa.TreeStep(cache.key, cache.value, cache.key_exps, cache.value_exps, batch=1,
                                     num_heads=2, max_seqlen_q=1, max_blocks_per_seq=1)):
        with pytest.raises(pa.PaError, match="CUDA device"):
            call()


def test_a_cache_is_freed_with_its_last_name():
    import weakref
    cache = pa.QuantCache.empty(2, 16, 2, 64, device="cpu")
    cache._configs[1, 1, 1]
    codes = weakref.ref(cache.key)
    del cache
    assert codes() is None


@pytest.mark.parametrize("call", ["rotate", "write", "store", "read"])
def test_a_configuration_lives_as_long_as_its_call(monkeypatch, call):
    """While the C side has a configuration's address, another thread's new
    configurations may clear the dictionary that holds it."""
    import weakref

    from paged_kv_cache_206_gb300 import serving
    cache = pa.QuantCache.empty(2, 16, 2, 64, device="cpu")
    rows, ints = torch.zeros((1, 2, 64), dtype=torch.float16), torch.ones(1, dtype=torch.int32)
    table, out = torch.zeros((1, 1), dtype=torch.int32), torch.zeros((1, 2, 64), dtype=torch.float16)
    serving._rotations.clear()
    calls = []

    def launch(where, at, stream, function, *args):
        held = [c for d in (cache._configs, serving._rotations) for c in d.values()]
        used = [weakref.ref(c) for a, c in held if a in args]
        del held
        cache._configs.clear()
        serving._rotations.clear()
        calls.append(len(used))
        assert all(c() is not None for c in used)

    monkeypatch.setattr(serving, "_launch", launch)
    if call == "rotate":
        pa.pa_qk_norm_rope(rows, rows, None, None, None, ints, out, out.clone())
    elif call == "write":
        cache.write(rows, rows, table, ints)
    elif call == "store":
        cache.store(rows, rows, rows, None, None, None, None, table, ints, None, 1, out)
    else:
        cache.read(table, None, ints, torch.zeros_like(ints), 1, out, rows)
    assert calls == [2 if call == "store" else 1]


def test_the_build_does_without_pythons_headers(monkeypatch, tmp_path, lib):
    """The library is built (and a module of other sources taken away) where there is no Python.h."""
    called = tmp_path / "pa_call.so"
    called.write_bytes(b"")
    monkeypatch.setattr(build_lib, "CALL", str(called))
    monkeypatch.setattr(build_lib.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert build_lib.build() == build_lib.LIB
    assert not called.exists()


def test_the_module_is_named_for_its_interpreter():
    import sysconfig
    assert build_lib.CALL.endswith(sysconfig.get_config_var("EXT_SUFFIX"))


@pytest.mark.parametrize("module", [True, False])
def test_calls_with_and_without_the_module(monkeypatch, lib, module):
    """Both ways reach the library with every argument in its place."""
    from paged_kv_cache_206_gb300 import serving
    monkeypatch.setattr(serving, "_f16", None)
    if not module:
        monkeypatch.setattr(build_lib, "CALL", "/nonexistent")
    serving._start()
    assert (serving._call is serving._ctypes_call) == (not module)
    config = cache()

    def read(rows, k_out, v_out):
        return serving._call(serving._read, ctypes.addressof(config), FAKE.value, FAKE.value, OTHER.value,
                             OTHER.value, FAKE.value, None, FAKE.value, FAKE.value, rows, k_out, v_out, None, 0)
    assert read(0, FAKE.value, OTHER.value) == pa.PA_OK
    assert read(-1, FAKE.value, OTHER.value) == pa.PA_ERR_INVALID_ARG
    assert read(0, FAKE.value, FAKE.value) == pa.PA_ERR_INVALID_ARG
    assert read(0, FAKE.value, BAD.value) == pa.PA_ERR_INVALID_ARG
    monkeypatch.undo()
    serving._start()


@pytest.mark.parametrize("tokens", [2**31, 2**58, 2**60, 2**61, 2**62, 2**63 - 1])
def test_numbers_of_tokens_whose_products_pass_64_bits_are_refused(lib, tokens):
    """Before anything is launched: on a machine without a GPU a launch would be PA_ERR_CUDA."""
    assert call_rotate(lib, tokens=tokens) == pa.PA_ERR_INVALID_ARG
    assert call_rotate(lib, rotary(num_heads=8, kv_heads=8), tokens=tokens, qs=512, ks=512) == pa.PA_ERR_INVALID_ARG
    assert call_write(lib, tokens=tokens) == pa.PA_ERR_INVALID_ARG
    assert call_write(lib, store=rotary(), tokens=tokens) == pa.PA_ERR_INVALID_ARG
    for heads in (8, 32):
        for d in (64, 128, 272):
            cfg = tree_cfg(num_heads=heads, head_size_k=d)
            assert lib.pa_tree_forward(ctypes.byref(cfg), tokens, FAKE, FAKE, OTHER, None, None, FAKE, FAKE, FAKE,
                                       FAKE, FAKE, 1 << 40, OTHER, None) == pa.PA_ERR_INVALID_ARG
