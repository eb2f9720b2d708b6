"""Binding of the calls around the attention: include/pa_cache.h (norm and
rotation of queries and keys, the 8-bit cache written and read back) and
include/pa_tree.h (attention for drafted tokens over either cache).

The functions check what the C side cannot see (types, shapes, strides, the
device), marshal, and raise :class:`PaError`. They allocate nothing and launch
on the tensors' device, on ``stream`` or that device's current stream.
"""
from __future__ import annotations

import ctypes

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


def _launch(where, device, stream, call):
    """``call(stream handle)`` with the tensors' device current."""
    import torch
    if device.type != "cuda":
        _refuse(where, f"tensors must be on a CUDA device, got {device}")
    if stream is not None:
        if stream.device != device:
            _refuse(where, f"the stream is on {stream.device}, the tensors on {device}")
        handle = stream.cuda_stream
    else:
        handle = torch._C._cuda_getCurrentRawStream(device.index)
    if torch.cuda.current_device() == device.index:
        status = call(handle)
    else:
        with torch.cuda.device(device):
            status = call(handle)
    if status:
        _check(status, where)


def _status_arg(where, status, device):
    if status is None:
        return None
    import torch
    if status.numel() < 1 or status.element_size() != 4 or status.device != device \
            or status.dtype not in (torch.int32, torch.uint32):
        _refuse(where, "status must be an int32 or uint32 tensor of one element on the device")
    return status.data_ptr()


def _rotary(where, query, q_weight, k_weight, cos_sin, positions, q_out, kv_heads, eps, interleaved,
            device):
    """Checks of the rotation's arguments; its config."""
    f16, i32, f32, _, _ = _dtypes()
    tokens, heads, size = query.shape
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _dense(where, name, w, f16, device, (size,))
    rot, limit = 0, 2**31 - 1
    if cos_sin is not None:
        if cos_sin.dim() != 2:
            _refuse(where, "cos_sin must be [max_positions, rotary_dim]")
        _dense(where, "cos_sin", cos_sin, f32, device)
        limit, rot = cos_sin.shape
    if positions is not None:
        _dense(where, "positions", positions, i32, device, (tokens,))
    _dense(where, "q_out", q_out, f16, device, (tokens, heads, size))
    return pa_rotary(heads, kv_heads, size, rot, bool(interleaved), limit, eps)


def pa_qk_norm_rope(query, key, q_weight, k_weight, cos_sin, positions, q_out, k_out, eps=1e-6,
                    interleaved=False, status=None, stream=None) -> None:
    """Norm and rotate the heads of ``query`` [T, H, hk] and ``key`` [T, Hk, hk]
    (fp16; views into one packed projection will do) into ``q_out`` and
    ``k_out``, in one pass. ``q_weight`` / ``k_weight`` [hk] may be None (no
    norm); ``cos_sin`` is fp32 [max_positions, rotary_dim] (None: no rotation);
    ``positions`` int32 [T], -1 for padding tokens, which are left out."""
    where = "pa_qk_norm_rope"
    f16 = _dtypes()[0]
    if query.dim() != 3 or key.dim() != 3 or positions is None:
        _refuse(where, "query and key must be [tokens, heads, head_size], with positions")
    dev, tokens, size = query.device, query.shape[0], query.shape[2]
    kv_heads = key.shape[1]
    qs = _rows(where, "query", query, f16, dev, tokens, query.shape[1], size)
    ks = _rows(where, "key", key, f16, dev, tokens, kv_heads, size)
    rot = _rotary(where, query, q_weight, k_weight, cos_sin, positions, q_out, kv_heads, eps,
                  interleaved, dev)
    _dense(where, "k_out", k_out, f16, dev, (tokens, kv_heads, size))
    if tokens == 0:
        return
    st = _status_arg(where, status, dev)
    lib = load_library()
    _launch(where, dev, stream, lambda s: lib.pa_qk_norm_rope(
        ctypes.byref(rot), tokens, query.data_ptr(), qs, key.data_ptr(), ks, _ptr(q_weight),
        _ptr(k_weight), _ptr(cos_sin), positions.data_ptr(), q_out.data_ptr(), k_out.data_ptr(), st, s))


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
        self.device = key.device

    @classmethod
    def empty(cls, num_blocks, block_size, kv_heads, head_size_k, head_size_v=None, device="cuda"):
        import torch
        hv = head_size_k if head_size_v is None else head_size_v
        codes = [torch.zeros((num_blocks, block_size, kv_heads, n), dtype=torch.float8_e4m3fn,
                             device=device) for n in (head_size_k, hv)]
        exps = [torch.zeros((num_blocks, kv_heads, block_size), dtype=torch.uint8, device=device)
                for _ in range(2)]
        return cls(*codes, *exps)

    def _config(self, block_tables, max_rows):
        nb, bs, heads, hk = self.key.shape
        batch, cols = block_tables.shape
        return pa_cache_config(batch, heads, hk, self.value.shape[3], bs, nb, cols, max_rows)

    def write(self, key, value, block_tables, context_lens, q_seqlens=None, max_seqlen_q=None,
              status=None, stream=None) -> None:
        """Quantise the current tokens' ``key`` [T, Hk, hk] and ``value``
        [T, Hk, hv] (fp16) into the cache (pa_cache_write)."""
        where, dev, f16 = "pa_cache_write", self.device, _dtypes()[0]
        if key.dim() != 3:
            _refuse(where, "key must be [tokens, kv_heads, head_size]")
        tokens, heads = key.shape[0], self.key.shape[2]
        ks = _rows(where, "key", key, f16, dev, tokens, heads, self.key.shape[3])
        vs = _rows(where, "value", value, f16, dev, tokens, heads, self.value.shape[3])
        _batch_args(where, block_tables, context_lens, q_seqlens, dev)
        if tokens == 0:
            return
        cfg = self._config(block_tables, tokens if max_seqlen_q is None else max_seqlen_q)
        st, lib = _status_arg(where, status, dev), load_library()
        _launch(where, dev, stream, lambda s: lib.pa_cache_write(
            ctypes.byref(cfg), tokens, key.data_ptr(), ks, value.data_ptr(), vs,
            block_tables.data_ptr(), context_lens.data_ptr(), _ptr(q_seqlens), self.key.data_ptr(),
            self.key_exps.data_ptr(), self.value.data_ptr(), self.value_exps.data_ptr(), st, s))

    def store(self, query, key, value, q_weight, k_weight, cos_sin, positions, block_tables,
              context_lens, q_seqlens, max_seqlen_q, q_out, eps=1e-6, interleaved=False, status=None,
              stream=None) -> None:
        """Norm and rotate ``query`` into ``q_out`` and ``key`` into the cache,
        with ``value``, in one pass (pa_cache_store). ``positions`` None takes
        the cache positions."""
        where, dev, f16 = "pa_cache_store", self.device, _dtypes()[0]
        if query.dim() != 3:
            _refuse(where, "query must be [tokens, heads, head_size]")
        tokens, heads, size = query.shape[0], self.key.shape[2], self.key.shape[3]
        qs = _rows(where, "query", query, f16, dev, tokens, query.shape[1], size)
        ks = _rows(where, "key", key, f16, dev, tokens, heads, size)
        vs = _rows(where, "value", value, f16, dev, tokens, heads, self.value.shape[3])
        rot = _rotary(where, query, q_weight, k_weight, cos_sin, positions, q_out, heads, eps,
                      interleaved, dev)
        _batch_args(where, block_tables, context_lens, q_seqlens, dev)
        if tokens == 0:
            return
        cfg = self._config(block_tables, tokens if max_seqlen_q is None else max_seqlen_q)
        st, lib = _status_arg(where, status, dev), load_library()
        _launch(where, dev, stream, lambda s: lib.pa_cache_store(
            ctypes.byref(cfg), ctypes.byref(rot), tokens, query.data_ptr(), qs, key.data_ptr(), ks,
            value.data_ptr(), vs, _ptr(q_weight), _ptr(k_weight), _ptr(cos_sin), _ptr(positions),
            block_tables.data_ptr(), context_lens.data_ptr(), _ptr(q_seqlens), self.key.data_ptr(),
            self.key_exps.data_ptr(), self.value.data_ptr(), self.value_exps.data_ptr(),
            q_out.data_ptr(), st, s))

    def read(self, block_tables, starts, context_lens, out_starts, max_rows, k_out, v_out,
             status=None, stream=None) -> None:
        """Read positions ``starts[b]`` (None: 0) up to ``context_lens[b]`` of every
        sequence back as fp16 rows from row ``out_starts[b]`` of ``k_out``
        [rows, Hk, hk] and ``v_out`` [rows, Hk, hv]; ``max_rows`` is the most rows
        of one sequence (pa_cache_read)."""
        where, dev = "pa_cache_read", self.device
        f16, i32, _, _, _ = _dtypes()
        rows, heads = k_out.shape[0], self.key.shape[2]
        _dense(where, "k_out", k_out, f16, dev, (rows, heads, self.key.shape[3]))
        _dense(where, "v_out", v_out, f16, dev, (rows, heads, self.value.shape[3]))
        _batch_args(where, block_tables, context_lens, starts, dev)
        _dense(where, "out_starts", out_starts, i32, dev, context_lens.shape)
        if rows == 0:
            return
        cfg = self._config(block_tables, max_rows)
        st, lib = _status_arg(where, status, dev), load_library()
        _launch(where, dev, stream, lambda s: lib.pa_cache_read(
            ctypes.byref(cfg), self.key.data_ptr(), self.key_exps.data_ptr(), self.value.data_ptr(),
            self.value_exps.data_ptr(), block_tables.data_ptr(), _ptr(starts),
            context_lens.data_ptr(), out_starts.data_ptr(), rows, k_out.data_ptr(), v_out.data_ptr(),
            st, s))


def pa_tree_workspace(cfg) -> int:
    """Bytes of workspace that pa_tree_forward needs for ``cfg``."""
    n = ctypes.c_size_t()
    _check(load_library().pa_tree_workspace(ctypes.byref(cfg), ctypes.byref(n)), "pa_tree_workspace")
    return n.value


class TreeStep:
    """Attention of drafted tokens (a tree, a chain, or one token per sequence)
    over a paged cache (pa_tree_forward). Holds the configuration and a
    workspace; a step's launches do not depend on the lengths, so :meth:`run`
    may be captured in a CUDA graph. ``key_exps`` and ``value_exps`` select the
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

    def run(self, query, block_tables, context_lens, q_seqlens, parents, out, stream=None):
        """Attend ``query`` [T, H, hk] into ``out`` [T, H, hv]; ``parents`` int32 [T]
        or None (a chain). Returns ``out``."""
        where, dev, cfg = "pa_tree_forward", self.device, self.cfg
        f16, i32, _, _, _ = _dtypes()
        tokens = query.shape[0]
        _dense(where, "query", query, f16, dev, (tokens, cfg.num_heads, cfg.head_size_k))
        _dense(where, "out", out, f16, dev, (tokens, cfg.num_heads, cfg.head_size_v))
        _batch_args(where, block_tables, context_lens, q_seqlens, dev)
        if block_tables.shape != (cfg.batch, cfg.max_blocks_per_seq):
            _refuse(where, f"block_tables must be [{cfg.batch}, {cfg.max_blocks_per_seq}]")
        if parents is not None:
            _dense(where, "parents", parents, i32, dev, (tokens,))
        if tokens == 0:
            return out
        lib, ws = load_library(), self.workspace
        _launch(where, dev, stream, lambda s: lib.pa_tree_forward(
            ctypes.byref(cfg), tokens, query.data_ptr(), self.key.data_ptr(), self.value.data_ptr(),
            _ptr(self.key_exps), _ptr(self.value_exps), block_tables.data_ptr(),
            context_lens.data_ptr(), _ptr(q_seqlens), _ptr(parents), ws.data_ptr(), ws.numel(),
            out.data_ptr(), s))
        return out

    def status(self, stream=None):
        return pa_status_read(self.workspace, stream)
