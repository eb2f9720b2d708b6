"""Plain references in 64 bits for the calls of pa_window.h and pa_blocks.h, and for positions
of several axes. numpy only; nothing here shares code with the library."""
import numpy as np


def sees(q, ctx, window, sinks):
    """Which of the ctx keys each of the q current tokens attends."""
    pos = np.arange(ctx - q, ctx)[:, None]
    key = np.arange(ctx)
    return (key <= pos) & ((key > pos - window) | (key < sinks))


def window_attention(query, key, value, value_exp, batch, window, sinks, scale, only=None):
    """(out, bound) of float64 caches [num_blocks, bs, Hk, d] (dequantised values; ``value_exp``
    [num_blocks, Hk, bs] the exponents of the value rows, zeros for an fp16 cache). Keys that a
    row does not attend may hold anything. ``only``: the sequences to compute.

    The bound on |fp16 result - out| counts, with p the weights and A = sum p |v|:
      2^-11 |out|  the result's rounding;
      2^-11 A      the weights' rounding to fp16 for the matrix product;
      2^-25 Pmax sum |codes|  that rounding where a weight is subnormal in fp16:
                   an absolute 2^-25 of the largest p 2^ev, for every key;
      2 A ds       a score off by ds: fp32 products and sums of hk terms, each
                   half a step of the terms' magnitudes, the factors applied to it, and
                   ex2.approx (2 steps); the weights and their sum both move.
    """
    H, hk, hv = query.shape[1], key.shape[3], value.shape[3]
    G = H // key.shape[2]
    out = np.zeros((query.shape[0], H, hv))
    bound = np.zeros_like(out)
    for b in range(len(batch.q)) if only is None else only:
        q, L, t0 = int(batch.q[b]), int(batch.ctx[b]), int(batch.starts[b])
        if q == 0:
            continue
        see = sees(q, L, window, sinks)
        keys = np.flatnonzero(see.any(0))
        see = see[:, keys]
        blk, off = batch.tables[b, keys // batch.block].astype(np.int64), keys % batch.block
        for h in range(H):
            k, v = key[blk, off, h // G], value[blk, off, h // G]
            ev = value_exp[blk, h // G, off].astype(np.float64)
            x = query[t0:t0 + q, h].astype(np.float64)
            s = scale * (x @ k.T)
            mag = np.where(see, scale * (np.abs(x) @ np.abs(k.T)), 0).max(1)
            s = np.where(see, s, -np.inf)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            o, A = p @ v, p @ np.abs(v)
            codes = see @ (np.abs(v) * 2.0 ** -ev[:, None])
            ds = ((hk + 8) * 2.0**-24 * mag + 2.0**-21)[:, None]
            pmax = (p * 2.0**ev).max(1)[:, None]
            out[t0:t0 + q, h] = o
            bound[t0:t0 + q, h] = (2.0**-11 * np.abs(o) + 2.0**-11 * A + 2 * A * ds + 2.0**-25 * pmax * codes
                                   + 2.0**-25)
    return out, bound


class Pool:
    """The pool of pa_blocks.h in lists."""

    def __init__(self, batch, cols, num_blocks, bs, window=0, sinks=0):
        self.tables = [[-1] * cols for _ in range(batch)]
        self.held, self.gone = [0] * batch, [0] * batch
        self.free, self.count = list(range(num_blocks - 1, -1, -1)), num_blocks
        self.cols, self.bs, self.window, self.kept = cols, bs, window, min(-(-sinks // bs), cols)

    def step(self, ctx, q, tokens):
        """(slots, positions, whether blocks ran out)."""
        lens = [(L, n if q is not None else 0) for L, n in zip(ctx, q if q is not None else ctx)]
        q_of = [n for _, n in lens] if q is not None else [1 if L > 0 else 0 for L in ctx]
        ok = [0 <= n <= L <= self.cols * self.bs for n, L in zip(q_of, ctx)]
        back = []
        for b, L in enumerate(ctx):
            if not ok[b]:
                continue
            start = self.kept + self.gone[b]
            if L == 0:
                pages = [i for i in range(self.held[b]) if i < self.kept or i >= start]
            else:
                lo = max(0, L - q_of[b] - self.window + 1) if self.window else 0
                pages = list(range(start, min(lo // self.bs, self.held[b])))
                self.gone[b] += len(pages)
            for i in pages:
                back.append(self.tables[b][i])
                self.tables[b][i] = -1
            if L == 0:
                self.held[b] = self.gone[b] = 0
        for block in reversed(back):
            self.free[self.count] = block
            self.count += 1
        out_of = False
        for b, L in enumerate(ctx):
            while ok[b] and self.held[b] * self.bs < L:
                if self.count == 0:
                    out_of = True
                    break
                self.count -= 1
                self.tables[b][self.held[b]] = self.free[self.count]
                self.held[b] += 1
        slots, positions = [-1] * tokens, [-1] * tokens
        t = 0
        for b, L in enumerate(ctx):
            stated = max(q[b], 0) if q is not None else 1
            for i in range(q_of[b] if ok[b] else 0):
                if t + i >= tokens:
                    break
                p = L - q_of[b] + i
                positions[t + i] = p
                if p // self.bs < self.held[b] and self.tables[b][p // self.bs] >= 0:
                    slots[t + i] = self.tables[b][p // self.bs] * self.bs + p % self.bs
            t += stated
        return slots, positions, out_of


def axis_of_pair(sections, cyclic, pairs):
    axes, out = len(sections), []
    for i in range(pairs):
        if cyclic:
            a = i % axes
            out.append(a if a and i < axes * sections[a] else 0)
        else:
            out.append(next(a for a in range(axes) if i < sum(sections[:a + 1])))
    return out


def rotate_axes(x, weight, cos_sin, positions, sections, cyclic, eps, interleaved):
    """serving_ref.rotate with positions [axes, tokens]."""
    y = x.astype(np.float64)
    if weight is not None:
        y = y / np.sqrt((y**2).mean(-1, keepdims=True) + eps) * weight.astype(np.float64)
    out, mag = y.copy(), np.abs(y)
    rot = cos_sin.shape[1]
    t = cos_sin.astype(np.float64)
    for i, axis in enumerate(axis_of_pair(sections, cyclic, rot // 2)):
        c, s = t[positions[axis], i][:, None], t[positions[axis], rot // 2 + i][:, None]
        lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        a, b = y[..., lo], y[..., hi]
        out[..., lo], out[..., hi] = a * c - b * s, b * c + a * s
        mag[..., lo], mag[..., hi] = np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)
    return out, mag
