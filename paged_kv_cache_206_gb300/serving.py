"""Binding of the calls around the attention: include/pa_cache.h (norm and
rotation of queries and keys, the 8-bit cache written and read back) and
include/pa_tree.h (attention for drafted tokens over either cache).

The functions check what the C side cannot see (types, shapes, strides, the
device), marshal, and raise :class:`PaError`. They allocate nothing and launch
on the tensors' device, on ``stream`` or that device's current stream.
"""
from __future__ import annotations

import ctypes
import os

from . import (PA_ERR_INVALID_ARG, PA_MASK_NONE, PaError, _check, load_library, make_config,
               pa_status_read)


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


# A call first puts one question to its arguments, whether all are in order: a decode
# loop pays for that alone. Where the answer is no, the checks behind it say what is wrong.

_f16 = _i32 = _f32 = _stream = _device = _call = None
_rope = _write = _store = _read = _tree = None  # addresses of the library's functions


def _start():
    """torch's types, the calls that tell the current stream and device, the library's
    functions and what calls them."""
    global _f16, _i32, _f32, _stream, _device, _call, _rope, _write, _store, _read, _tree
    import importlib.util

    import torch

    from .build_lib import CALL
    _i32, _f32 = torch.int32, torch.float32
    _stream, _device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    lib = load_library()
    _rope, _write, _store, _read, _tree = (
        ctypes.cast(f, ctypes.c_void_p).value
        for f in (lib.pa_qk_norm_rope, lib.pa_cache_write, lib.pa_cache_store, lib.pa_cache_read,
                  lib.pa_tree_forward))
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


def _rotary(where, query, q_weight, k_weight, cos_sin, positions, q_out, device):
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
        _dense(where, "positions", positions, _i32, device, (tokens,))
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


def _rotary_ok(at, tokens, heads, size, q_weight, k_weight, cos_sin, positions, q_out):
    return (_ok(q_weight, _f16, at, (size,)) and _ok(k_weight, _f16, at, (size,))
            and _ok(positions, _i32, at, (tokens,)) and _ok(q_out, _f16, at, (tokens, heads, size))
            and (cos_sin is None or (cos_sin.dim() == 2 and _ok(cos_sin, _f32, at, cos_sin.shape))))


def _rot_config(heads, kv_heads, size, cos_sin, eps, interleaved):
    limit, rot = (2**31 - 1, 0) if cos_sin is None else cos_sin.shape
    return _rotations[heads, kv_heads, size, rot, 1 if interleaved else 0, limit, eps]


def pa_qk_norm_rope(query, key, q_weight, k_weight, cos_sin, positions, q_out, k_out, eps=1e-6,
                    interleaved=False, status=None, stream=None) -> None:
    """Norm and rotate the heads of ``query`` [T, H, hk] and ``key`` [T, Hk, hk]
    (fp16; views into one packed projection will do) into ``q_out`` and
    ``k_out``, in one pass. ``q_weight`` / ``k_weight`` [hk] may be None (no
    norm); ``cos_sin`` is fp32 [max_positions, rotary_dim] (None: no rotation);
    ``positions`` int32 [T], -1 for padding tokens, which are left out."""
    where = "pa_qk_norm_rope"
    if _f16 is None:
        _start()
    if query.dim() != 3 or key.dim() != 3 or positions is None:
        _refuse(where, "query and key must be [tokens, heads, head_size], with positions")
    tokens, heads, size = query.shape
    at, kv_heads = query.get_device(), key.shape[1]
    qs = _token_stride(query, at, tokens, heads, size)
    ks = _token_stride(key, at, tokens, kv_heads, size)
    if not (qs is not None and ks is not None and _ok(k_out, _f16, at, (tokens, kv_heads, size))
            and _rotary_ok(at, tokens, heads, size, q_weight, k_weight, cos_sin, positions, q_out)):
        dev = query.device
        qs = _rows(where, "query", query, _f16, dev, tokens, heads, size)
        ks = _rows(where, "key", key, _f16, dev, tokens, kv_heads, size)
        _rotary(where, query, q_weight, k_weight, cos_sin, positions, q_out, dev)
        _dense(where, "k_out", k_out, _f16, dev, (tokens, kv_heads, size))
    if tokens == 0:
        return
    rotation = _rot_config(heads, kv_heads, size, cos_sin, eps, interleaved)
    _launch(where, at, stream, _rope, rotation[0], tokens,
            query.data_ptr(), qs, key.data_ptr(), ks, _ptr(q_weight), _ptr(k_weight), _ptr(cos_sin),
            positions.data_ptr(), q_out.data_ptr(), k_out.data_ptr(),
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
              stream=None) -> None:
        """Norm and rotate ``query`` into ``q_out`` and ``key`` into the cache,
        with ``value``, in one pass (pa_cache_store). ``positions`` None takes
        the cache positions."""
        where, at, heads = "pa_cache_store", self._at, self._heads
        if query.dim() != 3:
            _refuse(where, "query must be [tokens, heads, head_size]")
        (tokens, qh, size), hk, hv = query.shape, self._hk, self._hv
        qs = _token_stride(query, at, tokens, qh, hk)
        ks = _token_stride(key, at, tokens, heads, hk)
        vs = _token_stride(value, at, tokens, heads, hv)
        if not (qs is not None and ks is not None and vs is not None
                and _rotary_ok(at, tokens, qh, hk, q_weight, k_weight, cos_sin, positions, q_out)
                and _batch_ok(at, block_tables, context_lens, q_seqlens)):
            dev = self.device
            qs = _rows(where, "query", query, _f16, dev, tokens, qh, hk)
            ks = _rows(where, "key", key, _f16, dev, tokens, heads, hk)
            vs = _rows(where, "value", value, _f16, dev, tokens, heads, hv)
            _rotary(where, query, q_weight, k_weight, cos_sin, positions, q_out, dev)
            _batch_args(where, block_tables, context_lens, q_seqlens, dev)
        if tokens == 0:
            return
        config = self._configs[(*block_tables.shape, tokens if max_seqlen_q is None else max_seqlen_q)]
        rotation = _rot_config(qh, heads, hk, cos_sin, eps, interleaved)
        _launch(where, at, stream, _store, config[0], rotation[0], tokens, query.data_ptr(),
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


class TreeStep:
    """Attention of drafted tokens (a tree, a chain, or one token per sequence)
    over a paged cache (pa_tree_forward). Holds the configuration and a
    workspace; a step's launches do not depend on the lengths, so :meth:`run`
    may be captured in a CUDA graph. Steps that overlap on the GPU need a TreeStep
    each; keep it until its work is done. ``key_exps`` and ``value_exps`` select the
    8-bit cache of :class:`QuantCache`, None the fp16 one."""

    def __init__(self, key, value, key_exps=None, value_exps=None, *, batch, num_heads,
                 max_seqlen_q, max_blocks_per_seq, scale=0.0):
        import torch
        where = "TreeStep"
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
        self.workspace = torch.zeros(pa_tree_workspace(self.cfg), dtype=torch.uint8,
                                     device=self.device)
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(self.device).synchronize()  # zeroed before any stream's step
        if _f16 is None:
            _start()
        self._at = key.get_device()
        self._shapes = (num_heads, hk), (num_heads, value.shape[3]), (batch, max_blocks_per_seq)
        self._caches = tuple(_ptr(t) for t in (key, value, key_exps, value_exps))
        self._space = ctypes.addressof(self.cfg), self.workspace.data_ptr(), self.workspace.numel()

    def run(self, query, block_tables, context_lens, q_seqlens, parents, out, stream=None):
        """Attend ``query`` [T, H, hk] into ``out`` [T, H, hv]; ``parents`` int32 [T]
        or None (a chain). Returns ``out``."""
        where, at, tokens = "pa_tree_forward", self._at, query.shape[0]
        (q, o, tables), (cfg, space, size) = self._shapes, self._space
        if not (_ok(query, _f16, at, (tokens, *q)) and _ok(out, _f16, at, (tokens, *o))
                and block_tables.shape == tables and _batch_ok(at, block_tables, context_lens, q_seqlens)
                and _ok(parents, _i32, at, (tokens,))):
            dev = self.device
            _dense(where, "query", query, _f16, dev, (tokens, *q))
            _dense(where, "out", out, _f16, dev, (tokens, *o))
            _batch_args(where, block_tables, context_lens, q_seqlens, dev)
            if block_tables.shape != tables:
                _refuse(where, f"block_tables must be {list(tables)}")
            if parents is not None:
                _dense(where, "parents", parents, _i32, dev, (tokens,))
        if tokens == 0:
            return out
        _launch(where, at, stream, _tree, cfg, tokens,
                query.data_ptr(), *self._caches, block_tables.data_ptr(), context_lens.data_ptr(),
                _ptr(q_seqlens), _ptr(parents), space, size, out.data_ptr())
        return out

    def status(self, stream=None):
        return pa_status_read(self.workspace, stream)
