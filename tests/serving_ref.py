"""Plain references in 64 bits for the calls of pa_cache.h and pa_tree.h, and
batches to run them on. numpy only; nothing here shares code with the library."""
from dataclasses import dataclass

import numpy as np

E_MIN = -32


# ---- the 8-bit element: every code's value, and the nearest one to a number

def _code_values():
    v = np.empty(128)
    for c in range(128):
        e, m = c >> 3, c & 7
        v[c] = m / 8 * 2.0**-6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
    v[127] = np.nan
    return v


CODES = _code_values()


def decode(codes):
    codes = codes.astype(np.int64)
    return np.where(codes & 128, -1.0, 1.0) * CODES[codes & 127]


def encode(x):
    """Nearest e4m3 code of float64 values of at most 448, ties to the even code."""
    a = np.abs(x)
    mids = (CODES[:126] + CODES[1:127]) / 2
    c = np.searchsorted(mids, a, side="left")  # a <= mid stays below
    tie = (c < 126) & (a == mids[np.minimum(c, 125)]) & (c & 1 == 1)
    c = np.where(tie, c + 1, c)
    c = np.where(np.isfinite(x), c, 127)
    sign = np.signbit(x) & np.isfinite(x)
    return (c + 128 * sign).astype(np.uint8)


def row_exponent(x):
    """Least e >= E_MIN with max |finite x| <= 448 * 2^e, by trying them."""
    top = np.where(np.isfinite(x), np.abs(x), 0).max(-1)
    e = np.full(top.shape, E_MIN)
    while True:
        more = top > 448 * 2.0**e
        if not more.any():
            return e
        e = e + more


def quantise(x):
    """(codes, exponents) of float64 rows."""
    e = row_exponent(x)
    with np.errstate(invalid="ignore"):  # the NaN of a row
        return encode(x * 2.0 ** -e[..., None]), e


def same_codes(got, want):
    """Equal, any NaN code for any other."""
    nan = (got & 127) == 127
    return np.array_equal(nan, (want & 127) == 127) and np.array_equal(got[~nan], want[~nan])


# ---- batches

@dataclass
class Batch:
    tables: np.ndarray
    ctx: np.ndarray
    q: np.ndarray
    block: int
    num_blocks: int

    @property
    def starts(self):
        return np.concatenate([[0], np.cumsum(self.q)[:-1]]).astype(np.int32)

    def slots(self, b, lo, hi):
        pos = np.arange(lo, hi)
        return self.tables[b, pos // self.block].astype(np.int64), pos % self.block


def make_batch(rng, q, ctx, block, extra_cols=1):
    q, ctx = np.asarray(q, np.int32), np.asarray(ctx, np.int32)
    need = -(-ctx // block)
    total = int(need.sum()) + 3
    order = rng.permutation(total).astype(np.int32)
    cols = int(max(need.max(), 1)) + extra_cols
    tables = rng.integers(0, total, size=(len(q), cols)).astype(np.int32)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n] = order[at:at + n]
        at += n
    return Batch(tables, ctx, q, block, total)


def trees(rng, q, kind):
    """Parents of every sequence's drafts, concatenated; None for a chain."""
    if kind == "chain":
        return None
    out = []
    for n in q:
        for i in range(n):
            if kind == "roots":
                p = -1
            elif kind == "line":
                p = i - 1
            elif kind == "star":
                p = -1 if i == 0 else 0
            else:
                p = -1 if i == 0 or rng.random() < 0.15 else int(rng.integers(max(0, i - 5), i))
            out.append(p)
    return np.asarray(out, np.int32)


def sees(q, parents_of_seq):
    """Which drafts each draft attends."""
    m = np.zeros((q, q), bool)
    for i in range(q):
        j = i
        while j >= 0:
            m[i, j] = True
            j = j - 1 if parents_of_seq is None else int(parents_of_seq[j])
    return m


# ---- the operators

def rotate(x, weight, cos_sin, positions, eps, interleaved):
    """(rows, sum of the magnitudes added up in each element)."""
    y = x.astype(np.float64)
    if weight is not None:
        y = y / np.sqrt((y**2).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)
    out, mag = y.copy(), np.abs(y)
    if cos_sin is None:
        return out, mag
    rot = cos_sin.shape[1]
    t = cos_sin.astype(np.float64)[positions][:, None]
    c, s = t[..., :rot // 2], t[..., rot // 2:]
    lo = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    hi = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    a, b = y[..., lo], y[..., hi]
    out[..., lo], out[..., hi] = a * c - b * s, b * c + a * s
    mag[..., lo] = np.abs(a * c) + np.abs(b * s)
    mag[..., hi] = np.abs(b * c) + np.abs(a * s)
    return out, mag


def rotate_error(mag, dims):
    """Bound on the fp32 error of a rotated row, before its rounding: the sum
    of squares accumulates dims terms (at most dims half steps of fp32, halved by
    the root), and root, division, two products, the turn and its sum round
    about a dozen times."""
    return mag * (dims / 2 + 12) * 2.0**-24


def tree_attention(query, key, value, key_exp, value_exp, batch, parents, scale):
    """(out, bound) of float64 caches [num_blocks, bs, Hk, d]: dequantised
    values in ``key`` and ``value``; exponents of the value rows in
    ``value_exp`` (zeros for an fp16 cache).

    The bound on |fp16 result - out| counts, with p the weights and
    A = sum p |v|:
      2^-11 |out|  the result's rounding;
      2^-11 A      the weights' rounding to fp16 for the matrix product;
      2^-25 Pmax sum |codes|  that rounding where a weight is subnormal in fp16:
                   an absolute 2^-25 of the largest p 2^ev, for every key;
      2 A ds       a score off by ds: fp32 products and sums of hk terms, each
                   half a step of the terms' magnitudes, the factors applied to it, and
                   ex2.approx (2 steps); the weights and their sum both move.
    """
    H, hk, hv = query.shape[1], key.shape[3], value.shape[3]
    kv_heads = key.shape[2]
    G = H // kv_heads
    out = np.zeros((query.shape[0], H, hv))
    bound = np.zeros_like(out)
    for b in range(len(batch.q)):
        q, L, t0 = int(batch.q[b]), int(batch.ctx[b]), int(batch.starts[b])
        if q == 0:
            continue
        blk, off = batch.slots(b, 0, L)
        see = np.zeros((q, L), bool)
        see[:, :L - q] = True
        see[:, L - q:] = sees(q, None if parents is None else parents[t0:t0 + q])
        for h in range(H):
            k, v = key[blk, off, h // G], value[blk, off, h // G]
            ev = value_exp[blk, h // G, off].astype(np.float64)
            x = query[t0:t0 + q, h].astype(np.float64)
            for i in range(q):
                m = see[i]
                s = scale * (k[m] @ x[i])
                mag = (scale * (np.abs(k[m]) @ np.abs(x[i]))).max()
                p = np.exp(s - s.max())
                p /= p.sum()
                out[t0 + i, h] = p @ v[m]
                A = p @ np.abs(v[m])
                pv = p * 2.0 ** ev[m]
                codes = (np.abs(v[m]) * 2.0 ** -ev[m][:, None]).sum(0)
                ds = (hk + 8) * 2.0**-24 * mag + 2.0**-21
                bound[t0 + i, h] = (2.0**-11 * np.abs(out[t0 + i, h]) + 2.0**-11 * A + 2 * A * ds
                                    + 2.0**-25 * pv.max() * codes + 2.0**-25)
    return out, bound
