"""Binding of the calls around the attention: include/pa_cache.h (norm and
rotation of queries and keys, the 8-bit cache written and read back),
include/pa_tree.h (attention for drafted tokens over either cache),
include/pa_window.h (attention with a sliding window and sinks) and
include/pa_blocks.h (the blocks of a cache handed out and given back).

The functions check what the C side cannot see (types, shapes, strides, the
device), marshal, and raise :class:`PaError`. They allocate nothing and launch
on the tensors' device, on ``stream`` or that device's current stream.
"""
from __future__ import annotations

import ctypes
import os

from . import (PA_ERR_INVALID_ARG, PA_MASK_NONE, PA_MAX_AXES, PaError, _check, load_library,
               make_config, pa_status_read)


class pa_rotary(ctypes.Structure):
    """Mirror of ``pa_rotary`` in include/pa_cache.h."""

    _fields_ = [(n, ctypes.c_int32) for n in ("num_heads", "kv_heads", "head_size", "rotary_dim",
                                              "interleaved", "max_positions")]
    _fields_ += [("eps", ctypes.c_float)]


class pa_cache_config(ctypes.Structure):
    """Mirror of ``pa_cache_config`` in include/pa_cache.h."""

    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "kv_heads", "head_size_k", "head_size_v",
                                              "block_size", "num_blocks", "max_blocks_per_seq",
                                              "max_rows")]


class pa_axes(ctypes.Structure):
    """Mirror of ``pa_axes`` in include/pa_cache.h."""

    _fields_ = [("count", ctypes.c_int32), ("cyclic", ctypes.c_int32),
                ("sections", ctypes.c_int32 * PA_MAX_AXES)]


class pa_window(ctypes.Structure):
    """Mirror of ``pa_window`` in include/pa_window.h."""

    _fields_ = [(n, ctypes.c_int32) for n in ("window", "sinks")]


class pa_blocks_config(ctypes.Structure):
    """Mirror of ``pa_blocks_config`` in include/pa_blocks.h."""

    _fields_ = [(n, ctypes.c_int32) for n in ("batch", "block_size", "num_blocks",
                                              "max_blocks_per_seq", "window", "sinks")]


# A call first puts one question to its arguments, whether all are in order: a decode
# loop pays for that alone. Where the answer is no, the checks behind it say what is wrong.

_f16 = _i32 = _i64 = _f32 = _stream = _device = _call = None
# addresses of the library's functions
_rope = _write = _store = _read = _tree = _rope_axes = _store_axes = _window = _blocks = None


def _start():
    """torch's types, the calls that tell the current stream and device, the library's
    functions and what calls them."""
    global _f16, _i32, _i64, _f32, _stream, _device, _call, _rope, _write, _store, _read, _tree
    global _rope_axes, _store_axes, _window, _blocks
    import importlib.util

    import torch

    from .build_lib import CALL
    _i32, _i64, _f32 = torch.int32, torch.int64, torch.float32
    _stream, _device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    lib = load_library()
    _rope, _write, _store, _read, _tree, _rope_axes, _store_axes, _window, _blocks = (
        ctypes.cast(f, ctypes.c_void_p).value
        for f in (lib.pa_qk_norm_rope, lib.pa_cache_write, lib.pa_cache_store, lib.pa_cache_read,
                  lib.pa_tree_forward, lib.pa_qk_norm_rope_axes, lib.pa_cache_store_axes,
                  lib.pa_window_forward, lib.pa_blocks_step))
    if os.path.exists(CALL):
        spec = importlib.util.spec_from_file_location("pa_call", CALL)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        _call = module.call
    else:  # built without Python's headers
        _call = _ctypes_call
    _f16 = torch.float16


def _ctypes_call(address, *args):
    """What csrc/pa_call.c does, 3 to 5 us slower."""
    words = [None if a is None else a & (2**64 - 1) for a in args]
    return ctypes.CFUNCTYPE(ctypes.c_int, *[ctypes.c_void_p] * len(args))(address)(*words)


class _Configs(dict):
    """Configurations, each with its address, by their values: making one takes as long as
    the launch. A call keeps the pair by a name of its own until it returns: another thread
    may clear the dictionary meanwhile, and the address alone keeps nothing alive."""

    def __init__(self, kind):
        self.kind = kind

    def __missing__(self, values):
        if len(self) >= 4096:
            self.clear()
        struct = self.kind(*values)
        got = self[values] = ctypes.addressof(struct), struct
        return got


_rotations = _Configs(pa_rotary)


def _make_axes(cyclic, *sections):
    return pa_axes(len(sections), cyclic, (ctypes.c_int32 * PA_MAX_AXES)(*sections))


_axes = _Configs(_make_axes)


def _refuse(where: str, what: str):
    raise PaError(PA_ERR_INVALID_ARG, f"{where}: {what}")


def _dtypes():
    import torch
    return torch.float16, torch.int32, torch.float32, torch.uint8, torch.float8_e4m3fn


def _ptr(t):
    return None if t is None else t.data_ptr()


def _dense(where, name, t, dtype, device, shape=None):
    """A contiguous tensor of this type on this device (and of this shape)."""
    if t.dtype is not dtype or t.device != device or not t.is_contiguous():
        _refuse(where, f"{name} must be a contiguous {dtype} tensor on {device}, got {t.dtype} on "
                       f"{t.device}, strides {tuple(t.stride())}")
    if shape is not None and t.shape != shape:
        _refuse(where, f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")


def _rows(where, name, t, dtype, device, tokens, heads, size):
    """A row tensor [tokens, heads, size] whose heads are dense; its token stride."""
    if t.dtype is not dtype or t.device != device or t.shape != (tokens, heads, size):
        _refuse(where, f"{name} must be a {dtype} tensor [{tokens}, {heads}, {size}] on {device}, "
                       f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    st, sh, sd = t.stride()
    if (size > 1 and sd != 1) or (heads > 1 and sh != size):
        _refuse(where, f"{name}: the heads of a token must be contiguous, strides {tuple(t.stride())}")
    return st if tokens > 1 else heads * size


def _launch(where, at, stream, function, *args):
    """``function(*args, stream handle)`` with device ``at`` (the tensors') current."""
    if at < 0:
        _refuse(where, "tensors must be on a CUDA device")
    if stream is None:
        handle = _stream(at)
    elif stream.device.index == at:
        handle = stream.cuda_stream
    else:
        _refuse(where, f"the stream is on {stream.device}, the tensors on cuda:{at}")
    if _device() == at:
        status = _call(function, *args, handle)
    else:
        import torch
        with torch.cuda.device(at):
            status = _call(function, *args, handle)
    if status:
        _check(status, where)


def _status_arg(where, status, device):
    import torch
    if status.numel() < 1 or status.element_size() != 4 or status.device != device \
            or status.dtype not in (torch.int32, torch.uint32):
        _refuse(where, "status must be an int32 or uint32 tensor of one element on the device")
    return status.data_ptr()


def _axes_of(where, sections, cyclic, positions):
    """The configuration of positions [axes, tokens] whose pairs are divided into ``sections``."""
    if positions is None:
        _refuse(where, "positions of several axes must be given")
    got = _axes.get((cyclic, *sections))
    if got is not None:
        return got
    if not 1 <= len(sections) <= PA_MAX_AXES:
        _refuse(where, f"sections must be those of 1 to {PA_MAX_AXES} axes, got {tuple(sections)}")
    if any(not 0 <= int(s) < 2**31 for s in sections):
        _refuse(where, f"sections must be numbers of pairs, got {tuple(sections)}")
    return _axes[(1 if cyclic else 0, *map(int, sections))]


def _rotary(where, query, q_weight, k_weight, cos_sin, positions, q_out, device, places):
    """Checks of the rotation's arguments."""
    tokens, heads, size = query.shape
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _dense(where, name, w, _f16, device, (size,))
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            _refuse(where, "cos_sin must be [max_positions, rotary_dim]")
        _dense(where, "cos_sin", cos_sin, _f32, device)
    if positions is not None:
        _dense(where, "positions", positions, _i32, device, places)
    _dense(where, "q_out", q_out, _f16, device, (tokens, heads, size))


def _ok(t, dtype, at, shape):
    """Whether a tensor (or None) is dense, of this type and shape, on device ``at``."""
    return t is None or (t.dtype is dtype and t.get_device() == at and t.shape == shape
                         and t.is_contiguous())


def _token_stride(t, at, tokens, heads, size):
    """The token stride of fp16 rows [tokens, heads, size] with dense heads; None: they are not."""
    if t.dtype is _f16 and t.get_device() == at and t.shape == (tokens, heads, size):
        st, sh, sd = t.stride()
        if sh == size and sd == 1:
            return st if tokens > 1 else heads * size
    return None


def _rotary_ok(at, tokens, heads, size, q_weight, k_weight, cos_sin, positions, q_out, places):
    return (_ok(q_weight, _f16, at, (size,)) and _ok(k_weight, _f16, at, (size,))
            and _ok(positions, _i32, at, places) and _ok(q_out, _f16, at, (tokens, heads, size))
            and (cos_sin is None or (cos_sin.dim() == 2 and _ok(cos_sin, _f32, at, cos_sin.shape))))


def _rot_config(heads, kv_heads, size, cos_sin, eps, interleaved):
    limit, rot = (2**31 - 1, 0) if cos_sin is None else cos_sin.shape
    return _rotations[heads, kv_heads, size, rot, 1 if interleaved else 0, limit, eps]


def pa_qk_norm_rope(query, key, q_weight, k_weight, cos_sin, positions, q_out, k_out, eps=1e-6,
                    interleaved=False, status=None, stream=None, sections=None, cyclic=False) -> None:
    """Norm and rotate the heads of ``query`` [T, H, hk] and ``key`` [T, Hk, hk]
    (fp16; views into one packed projection will do) into ``q_out`` and
    ``k_out``, in one pass. ``q_weight`` / ``k_weight`` [hk] may be None (no
    norm); ``cos_sin`` is fp32 [max_positions, rotary_dim] (None: no rotation);
    ``positions`` int32 [T], -1 for padding tokens, which are left out.

    ``sections`` (pairs of each of up to four axes, rotary_dim / 2 together) makes
    ``positions`` int32 [axes, T]: pair i turns by the position of its axis, the axes'
    pairs lying behind one another, or in turn (``cyclic``; include/pa_cache.h)."""
    where = "pa_qk_norm_rope"
    if _f16 is None:
        _start()
    if query.dim() != 3 or key.dim() != 3 or positions is None:
        _refuse(where, "query and key must be [tokens, heads, head_size], with positions")
    tokens, heads, size = query.shape
    at, kv_heads = query.get_device(), key.shape[1]
    axes = None if sections is None else _axes_of(where, sections, cyclic, positions)
    places = (tokens,) if axes is None else (len(sections), tokens)
    qs = _token_stride(query, at, tokens, heads, size)
    ks = _token_stride(key, at, tokens, kv_heads, size)
    if not (qs is not None and ks is not None and _ok(k_out, _f16, at, (tokens, kv_heads, size))
            and _rotary_ok(at, tokens, heads, size, q_weight, k_weight, cos_sin, positions, q_out,
                           places)):
        dev = query.device
        qs = _rows(where, "query", query, _f16, dev, tokens, heads, size)
        ks = _rows(where, "key", key, _f16, dev, tokens, kv_heads, size)
        _rotary(where, query, q_weight, k_weight, cos_sin, positions, q_out, dev, places)
        _dense(where, "k_out", k_out, _f16, dev, (tokens, kv_heads, size))
    if tokens == 0:
        return
    rotation = _rot_config(heads, kv_heads, size, cos_sin, eps, interleaved)
    call = (_rope, rotation[0]) if axes is None else (_rope_axes, rotation[0], axes[0])
    _launch(where, at, stream, *call, tokens, query.data_ptr(), qs, key.data_ptr(), ks, _ptr(q_weight),
            _ptr(k_weight), _ptr(cos_sin), positions.data_ptr(), q_out.data_ptr(), k_out.data_ptr(),
            None if status is None else _status_arg(where, status, query.device))


def _cache_tensors(where, key, value, key_exps, value_exps):
    """Checks of a cache's tensors (fp16 without exponents, e4m3 with them)."""
    f16, _, _, u8, e4m3 = _dtypes()
    if key.dim() != 4 or value.dim() != 4 or key.shape[:3] != value.shape[:3]:
        _refuse(where, "the caches must be [num_blocks, block_size, kv_heads, head_size], alike but "
                       "for the head size")
    if (key_exps is None) != (value_exps is None):
        _refuse(where, "give the exponents of both caches or of neither")
    kind = f16 if key_exps is None else e4m3
    nb, bs, hk, _ = key.shape
    _dense(where, "key cache", key, kind, key.device)
    _dense(where, "value cache", value, kind, key.device)
    if key_exps is not None:
        _dense(where, "key_exps", key_exps, u8, key.device, (nb, hk, bs))
        _dense(where, "value_exps", value_exps, u8, key.device, (nb, hk, bs))


def _batch_ok(at, block_tables, context_lens, q_seqlens):
    shape = block_tables.shape
    return (len(shape) == 2 and _ok(block_tables, _i32, at, shape)
            and _ok(context_lens, _i32, at, shape[:1]) and _ok(q_seqlens, _i32, at, shape[:1]))


def _batch_args(where, block_tables, context_lens, q_seqlens, device):
    i32 = _dtypes()[1]
    if block_tables.dim() != 2:
        _refuse(where, "block_tables must be [batch, max_blocks_per_seq]")
    _dense(where, "block_tables", block_tables, i32, device)
    batch = (block_tables.shape[0],)
    _dense(where, "context_lens", context_lens, i32, device, batch)
    if q_seqlens is not None:
        _dense(where, "q_seqlens", q_seqlens, i32, device, batch)


class QuantCache:
    """A paged KV cache in 8 bits: e4m3 codes ``key`` and ``value``
    [num_blocks, block_size, kv_heads, head_size] with one exponent byte per
    token and kv head, ``key_exps`` and ``value_exps``
    [num_blocks, kv_heads, block_size] (include/pa_cache.h). The tensors are the
    caller's; :meth:`empty` makes them."""

    def __init__(self, key, value, key_exps, value_exps):
        if key_exps is None or value_exps is None:
            _refuse("QuantCache", "an 8-bit cache has exponents")
        _cache_tensors("QuantCache", key, value, key_exps, value_exps)
        self.key, self.value, self.key_exps, self.value_exps = key, value, key_exps, value_exps
        if _f16 is None:
            _start()
        self.device, self._at = key.device, key.get_device()
        nb, bs, heads, hk = key.shape
        hv = value.shape[3]
        self._heads, self._hk, self._hv = heads, hk, hv
        self._addresses = tuple(t.data_ptr() for t in (key, key_exps, value, value_exps))
        # (no reference to self: the caches are freed as soon as the last name of them is)
        self._configs = _Configs(lambda batch, cols, max_rows: pa_cache_config(
            batch, heads, hk, hv, bs, nb, cols, max_rows))

    @classmethod
    def empty(cls, num_blocks, block_size, kv_heads, head_size_k, head_size_v=None, device="cuda"):
        import torch
        hv = head_size_k if head_size_v is None else head_size_v
        codes = [torch.zeros((num_blocks, block_size, kv_heads, n), dtype=torch.float8_e4m3fn,
                             device=device) for n in (head_size_k, hv)]
        exps = [torch.zeros((num_blocks, kv_heads, block_size), dtype=torch.uint8, device=device)
                for _ in range(2)]
        return cls(*codes, *exps)

    def write(self, key, value, block_tables, context_lens, q_seqlens=None, max_seqlen_q=None,
              status=None, stream=None) -> None:
        """Quantise the current tokens' ``key`` [T, Hk, hk] and ``value``
        [T, Hk, hv] (fp16) into the cache (pa_cache_write)."""
        where, at, heads = "pa_cache_write", self._at, self._heads
        if key.dim() != 3:
            _refuse(where, "key must be [tokens, kv_heads, head_size]")
        tokens = key.shape[0]
        ks = _token_stride(key, at, tokens, heads, self._hk)
        vs = _token_stride(value, at, tokens, heads, self._hv)
        if not (ks is not None and vs is not None
                and _batch_ok(at, block_tables, context_lens, q_seqlens)):
            ks = _rows(where, "key", key, _f16, self.device, tokens, heads, self._hk)
            vs = _rows(where, "value", value, _f16, self.device, tokens, heads, self._hv)
            _batch_args(where, block_tables, context_lens, q_seqlens, self.device)
        if tokens == 0:
            return
        config = self._configs[(*block_tables.shape, tokens if max_seqlen_q is None else max_seqlen_q)]
        _launch(where, at, stream, _write, config[0],
                tokens, key.data_ptr(), ks, value.data_ptr(), vs, block_tables.data_ptr(),
                context_lens.data_ptr(), _ptr(q_seqlens), *self._addresses,
                None if status is None else _status_arg(where, status, self.device))

    def store(self, query, key, value, q_weight, k_weight, cos_sin, positions, block_tables,
              context_lens, q_seqlens, max_seqlen_q, q_out, eps=1e-6, interleaved=False, status=None,
              stream=None, sections=None, cyclic=False) -> None:
        """Norm and rotate ``query`` into ``q_out`` and ``key`` into the cache,
        with ``value``, in one pass (pa_cache_store). ``positions`` None takes
        the cache positions; with ``sections`` they have several axes (see
        :func:`pa_qk_norm_rope`) and are given."""
        where, at, heads = "pa_cache_store", self._at, self._heads
        if query.dim() != 3:
            _refuse(where, "query must be [tokens, heads, head_size]")
        (tokens, qh, size), hk, hv = query.shape, self._hk, self._hv
        axes = None if sections is None else _axes_of(where, sections, cyclic, positions)
        places = (tokens,) if axes is None else (len(sections), tokens)
        qs = _token_stride(query, at, tokens, qh, hk)
        ks = _token_stride(key, at, tokens, heads, hk)
        vs = _token_stride(value, at, tokens, heads, hv)
        if not (qs is not None and ks is not None and vs is not None
                and _rotary_ok(at, tokens, qh, hk, q_weight, k_weight, cos_sin, positions, q_out,
                               places)
                and _batch_ok(at, block_tables, context_lens, q_seqlens)):
            dev = self.device
            qs = _rows(where, "query", query, _f16, dev, tokens, qh, hk)
            ks = _rows(where, "key", key, _f16, dev, tokens, heads, hk)
            vs = _rows(where, "value", value, _f16, dev, tokens, heads, hv)
            _rotary(where, query, q_weight, k_weight, cos_sin, positions, q_out, dev, places)
            _batch_args(where, block_tables, context_lens, q_seqlens, dev)
        if tokens == 0:
            return
        config = self._configs[(*block_tables.shape, tokens if max_seqlen_q is None else max_seqlen_q)]
        rotation = _rot_config(qh, heads, hk, cos_sin, eps, interleaved)
        call = (_store, config[0], rotation[0]) if axes is None else (_store_axes, config[0], rotation[0], axes[0])
        _launch(where, at, stream, *call, tokens, query.data_ptr(),
                qs, key.data_ptr(), ks, value.data_ptr(), vs, _ptr(q_weight), _ptr(k_weight),
                _ptr(cos_sin), _ptr(positions), block_tables.data_ptr(), context_lens.data_ptr(),
                _ptr(q_seqlens), *self._addresses, q_out.data_ptr(),
                None if status is None else _status_arg(where, status, self.device))

    def read(self, block_tables, starts, context_lens, out_starts, max_rows, k_out, v_out,
             status=None, stream=None) -> None:
        """Read positions ``starts[b]`` (None: 0) up to ``context_lens[b]`` of every
        sequence back as fp16 rows from row ``out_starts[b]`` of ``k_out``
        [rows, Hk, hk] and ``v_out`` [rows, Hk, hv]; ``max_rows`` is the most rows
        of one sequence (pa_cache_read)."""
        where, at, rows = "pa_cache_read", self._at, k_out.shape[0]
        if not (_ok(k_out, _f16, at, (rows, self._heads, self._hk))
                and _ok(v_out, _f16, at, (rows, self._heads, self._hv))
                and _batch_ok(at, block_tables, context_lens, starts)
                and _ok(out_starts, _i32, at, context_lens.shape)):
            dev = self.device
            _dense(where, "k_out", k_out, _f16, dev, (rows, self._heads, self._hk))
            _dense(where, "v_out", v_out, _f16, dev, (rows, self._heads, self._hv))
            _batch_args(where, block_tables, context_lens, starts, dev)
            _dense(where, "out_starts", out_starts, _i32, dev, context_lens.shape)
        if rows == 0:
            return
        config = self._configs[(*block_tables.shape, max_rows)]
        _launch(where, at, stream, _read, config[0], *self._addresses,
                block_tables.data_ptr(), _ptr(starts), context_lens.data_ptr(), out_starts.data_ptr(),
                rows, k_out.data_ptr(), v_out.data_ptr(),
                None if status is None else _status_arg(where, status, self.device))


def pa_tree_workspace(cfg) -> int:
    """Bytes of workspace that pa_tree_forward needs for ``cfg``."""
    n = ctypes.c_size_t()
    _check(load_library().pa_tree_workspace(ctypes.byref(cfg), ctypes.byref(n)), "pa_tree_workspace")
    return n.value


class _PagedStep:
    """What :class:`TreeStep` and :class:`WindowStep` hold: the caches, the configuration and a
    workspace."""

    def _set(self, where, key, value, key_exps, value_exps, batch, num_heads, max_seqlen_q,
             max_blocks_per_seq, scale, workspace_of):
        import torch
        _cache_tensors(where, key, value, key_exps, value_exps)
        self.key, self.value, self.key_exps, self.value_exps = key, value, key_exps, value_exps
        self.device = key.device
        if self.device.type != "cuda":
            _refuse(where, f"the caches must be on a CUDA device, got {self.device}")
        nb, bs, heads, hk = key.shape
        sms = torch.cuda.get_device_properties(self.device).multi_processor_count
        self.cfg = make_config(batch=batch, num_heads=num_heads, kv_heads=heads, head_size_k=hk,
                               head_size_v=value.shape[3], block_size=bs, num_blocks=nb,
                               max_blocks_per_seq=max_blocks_per_seq, max_seqlen_q=max_seqlen_q,
                               mask_type=PA_MASK_NONE, num_sms=sms, scale=scale)
        self.workspace = torch.zeros(workspace_of(self.cfg), dtype=torch.uint8, device=self.device)
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(self.device).synchronize()  # zeroed before any stream's step
        if _f16 is None:
            _start()
        self._at = key.get_device()
        self._shapes = (num_heads, hk), (num_heads, value.shape[3]), (batch, max_blocks_per_seq)
        self._caches = tuple(_ptr(t) for t in (key, value, key_exps, value_exps))
        self._space = ctypes.addressof(self.cfg), self.workspace.data_ptr(), self.workspace.numel()

    def _batch(self, where, query, block_tables, context_lens, q_seqlens, out):
        """The checks behind the question whether a step's arguments are in order."""
        (q, o, tables), dev, tokens = self._shapes, self.device, query.shape[0]
        _dense(where, "query", query, _f16, dev, (tokens, *q))
        _dense(where, "out", out, _f16, dev, (tokens, *o))
        _batch_args(where, block_tables, context_lens, q_seqlens, dev)
        if block_tables.shape != tables:
            _refuse(where, f"block_tables must be {list(tables)}")

    def status(self, stream=None):
        return pa_status_read(self.workspace, stream)


class TreeStep(_PagedStep):
    """Attention of drafted tokens (a tree, a chain, or one token per sequence)
    over a paged cache (pa_tree_forward). Holds the configuration and a
    workspace; a step's launches do not depend on the lengths, so :meth:`run`
    may be captured in a CUDA graph. Steps that overlap on the GPU need a TreeStep
    each; keep it until its work is done. ``key_exps`` and ``value_exps`` select the
    8-bit cache of :class:`QuantCache`, None the fp16 one."""

    def __init__(self, key, value, key_exps=None, value_exps=None, *, batch, num_heads,
                 max_seqlen_q, max_blocks_per_seq, scale=0.0):
        self._set("TreeStep", key, value, key_exps, value_exps, batch, num_heads, max_seqlen_q,
                  max_blocks_per_seq, scale, pa_tree_workspace)

    def run(self, query, block_tables, context_lens, q_seqlens, parents, out, stream=None):
        """Attend ``query`` [T, H, hk] into ``out`` [T, H, hv]; ``parents`` int32 [T]
        or None (a chain). Returns ``out``."""
        where, at, tokens = "pa_tree_forward", self._at, query.shape[0]
        (q, o, tables), (cfg, space, size) = self._shapes, self._space
        if not (_ok(query, _f16, at, (tokens, *q)) and _ok(out, _f16, at, (tokens, *o))
                and block_tables.shape == tables and _batch_ok(at, block_tables, context_lens, q_seqlens)
                and _ok(parents, _i32, at, (tokens,))):
            self._batch(where, query, block_tables, context_lens, q_seqlens, out)
            if parents is not None:
                _dense(where, "parents", parents, _i32, self.device, (tokens,))
        if tokens == 0:
            return out
        _launch(where, at, stream, _tree, cfg, tokens,
                query.data_ptr(), *self._caches, block_tables.data_ptr(), context_lens.data_ptr(),
                _ptr(q_seqlens), _ptr(parents), space, size, out.data_ptr())
        return out


def pa_window_workspace(cfg, win) -> int:
    """Bytes of workspace that pa_window_forward needs for ``cfg`` and ``win``."""
    n = ctypes.c_size_t()
    _check(load_library().pa_window_workspace(ctypes.byref(cfg), ctypes.byref(win), ctypes.byref(n)),
           "pa_window_workspace")
    return n.value


class WindowStep(_PagedStep):
    """Attention with a sliding window over a paged cache (pa_window_forward): a token
    attends itself, the ``window - 1`` tokens before it and the first ``sinks`` of its
    sequence. Decode steps, chains of drafts, prompts and parts of prompts, over the
    fp16 cache or (with ``key_exps`` and ``value_exps``) the 8-bit one. What holds of
    graphs, streams and overlapping steps is what holds of :class:`TreeStep`."""

    def __init__(self, key, value, key_exps=None, value_exps=None, *, batch, num_heads,
                 max_seqlen_q, max_blocks_per_seq, window, sinks=0, scale=0.0):
        if not (0 < window < 2**31 and 0 <= sinks < 2**31):
            _refuse("WindowStep", f"window must be positive and sinks not negative, got {window} and {sinks}")
        self.win = pa_window(window, sinks)
        self._set("WindowStep", key, value, key_exps, value_exps, batch, num_heads, max_seqlen_q,
                  max_blocks_per_seq, scale, lambda cfg: pa_window_workspace(cfg, self.win))
        self._space += (ctypes.addressof(self.win),)

    def run(self, query, block_tables, context_lens, q_seqlens, out, stream=None):
        """Attend ``query`` [T, H, hk] into ``out`` [T, H, hv]. Returns ``out``."""
        where, at, tokens = "pa_window_forward", self._at, query.shape[0]
        (q, o, tables), (cfg, space, size, win) = self._shapes, self._space
        if not (_ok(query, _f16, at, (tokens, *q)) and _ok(out, _f16, at, (tokens, *o))
                and block_tables.shape == tables
                and _batch_ok(at, block_tables, context_lens, q_seqlens)):
            self._batch(where, query, block_tables, context_lens, q_seqlens, out)
        if tokens == 0:
            return out
        _launch(where, at, stream, _window, cfg, win, tokens,
                query.data_ptr(), *self._caches, block_tables.data_ptr(), context_lens.data_ptr(),
                _ptr(q_seqlens), space, size, out.data_ptr())
        return out


class BlockPool:
    """The blocks of a paged cache, handed out and given back on the GPU
    (pa_blocks_step): int32 tensors ``block_tables`` [batch, max_blocks_per_seq], ``held``
    and ``gone`` [batch], ``free`` [num_blocks] and ``count`` [1], the caller's;
    :meth:`empty` makes them. With a ``window``, blocks behind the first ``sinks`` positions
    go back as soon as no token attends them any more. Steps of one pool must not
    overlap; a step may be captured in a CUDA graph."""

    def __init__(self, block_tables, held, gone, free, count, *, block_size, window=0, sinks=0):
        where = "BlockPool"
        if _f16 is None:
            _start()
        if block_tables.dim() != 2 or free.dim() != 1:
            _refuse(where, "block_tables must be [batch, max_blocks_per_seq] and free [num_blocks]")
        dev, (batch, cols) = block_tables.device, block_tables.shape
        for name, t, shape in (("block_tables", block_tables, (batch, cols)), ("held", held, (batch,)),
                               ("gone", gone, (batch,)), ("free", free, free.shape), ("count", count, (1,))):
            _dense(where, name, t, _i32, dev, shape)
        if not all(0 <= n < 2**31 for n in (block_size, window, sinks)):
            _refuse(where, f"block_size, window and sinks must not be negative, got {block_size}, {window}, "
                           f"{sinks}")
        if max(batch, cols, free.shape[0]) >= 2**31:  # (before they are cut to 32 bits)
            _refuse(where, f"a pool has fewer than 2^31 rows, entries a row and blocks, got {batch}, {cols}, "
                           f"{free.shape[0]}")
        self.block_tables, self.held, self.gone, self.free, self.count = block_tables, held, gone, free, count
        self.cfg = pa_blocks_config(batch, block_size, free.shape[0], cols, window, sinks)
        self.device, self._at, self._rows = dev, block_tables.get_device(), (batch,)
        self._cfg = ctypes.addressof(self.cfg)
        self._addresses = tuple(t.data_ptr() for t in (block_tables, held, gone, free, count))

    @classmethod
    def empty(cls, batch, max_blocks_per_seq, num_blocks, block_size, window=0, sinks=0, device="cuda"):
        """A pool whose blocks are all free, block 0 on top."""
        import torch
        tables = torch.full((batch, max_blocks_per_seq), -1, dtype=torch.int32, device=device)
        held, gone = (torch.zeros(batch, dtype=torch.int32, device=device) for _ in range(2))
        free = torch.arange(num_blocks - 1, -1, -1, dtype=torch.int32, device=device)
        count = torch.full((1,), num_blocks, dtype=torch.int32, device=device)
        return cls(tables, held, gone, free, count, block_size=block_size, window=window, sinks=sinks)

    def step(self, context_lens, q_seqlens=None, slots=None, positions=None, status=None,
             stream=None) -> None:
        """Bring the tables to ``context_lens`` (0: the request is done), and the current tokens'
        cache slots and positions into ``slots`` int64 [T] and ``positions`` int32 [T] (either may
        be None), -1 behind the last one."""
        where, at, rows = "pa_blocks_step", self._at, self._rows
        given = slots if slots is not None else positions
        shape = (0,) if given is None else given.shape
        if not (len(shape) == 1 and _ok(context_lens, _i32, at, rows) and _ok(q_seqlens, _i32, at, rows)
                and _ok(slots, _i64, at, shape) and _ok(positions, _i32, at, shape)):
            dev = self.device
            _dense(where, "context_lens", context_lens, _i32, dev, rows)
            if q_seqlens is not None:
                _dense(where, "q_seqlens", q_seqlens, _i32, dev, rows)
            if len(shape) != 1:
                _refuse(where, "slots and positions must be [tokens]")
            if slots is not None:
                _dense(where, "slots", slots, _i64, dev, shape)
            if positions is not None:
                _dense(where, "positions", positions, _i32, dev, shape)
        _launch(where, at, stream, _blocks, self._cfg, context_lens.data_ptr(), _ptr(q_seqlens),
                *self._addresses, shape[0], _ptr(slots), _ptr(positions),
                None if status is None else _status_arg(where, status, self.device))
