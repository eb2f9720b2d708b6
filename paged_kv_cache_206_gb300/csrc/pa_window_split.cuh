// How pa_window_forward's kernels divide a batch: the line of pa_tree_split.cuh, cut into equal
// pieces, with row tiles that see different keys.
//
// A row tile is TT = NR / G whole tokens of one (sequence, kv head), or, for a group of more than
// NR heads, NR of one token's (HP parts). Tile t's first token stands at position p0 = L - q +
// t TT, its last at p1, and it walks the chunks of CHUNK keys that any of its rows attends, UNIT /
// CHUNK to a unit: those of the sinks before the window, then those from the first row's window
// on up to p1. To the kernels it is a tile of a sequence that ends with its last token; what the first row's window
// has left behind is their only addition.
//
// On the line a tile takes a place for each key of [0, p1] but those between the sinks and its
// first row's window, and LEAD units' worth for what it costs besides:
//   K_t = p1 + 1 - max(0, p0 + 1 - window - sinks)
// so the places up to a tile are a polynomial of t and of the first tile that leaves keys out:
// a worker finds its tile by bisection, whatever the lengths. A piece's ends fall on units in
// proportion, s = floor(x U / K) for place x of K and U units. As U * UNIT >= K and a worker has
// UNIT places at least, every worker between a tile's first and last one gets a unit; the last
// one does since x < K, and the first one that gets none leaves the tile to the next.
#pragma once

#include "pa_tree_split.cuh"

namespace pa {

// A row tile of which one worker has the units [s0, s1): as TreeTile says it of the sequence up to the
// tile's last token (q tokens, L keys), and what its rows' windows leave out.
struct WindowTile : TreeTile {
  int lo, lo1;    // the first keys of the first and of the last row's window
  int far, skip;  // chunks of the sinks, then so many chunks are left out
  int token0;     // the first row's token

  // where the c-th chunk stands in the sequence
  __host__ __device__ __forceinline__ int chunk(int c) const { return c < far ? c : c + skip; }
  // the position of the first row's token
  __host__ __device__ __forceinline__ int first() const { return L - q + token0; }
  // The token of the n-th row: the first one's and (its place in the group + n) / group, as a product with
  // 2^32 / group, which is exact while that and the group stay below 2^16.
  __device__ __forceinline__ int token(const TreeParams& P, int n) const {
    const int at = r0 - token0 * P.group + n;
    return token0 + (P.group_inverse ? int(__umulhi(uint32_t(at), P.group_inverse)) : at / P.group);
  }
};

// Whether none of the keys [key, key + n) is attended by a tile's rows, the first one's window beginning at lo.
__device__ __forceinline__ bool window_hidden(const TreeParams& P, int lo, int key, int n) {
  return key >= P.sinks && key + n <= lo;
}

// Whether the token at position p attends a key.
__device__ __forceinline__ bool window_sees(const TreeParams& P, int p, int key) {
  return key <= p && (p - key < P.window || key < P.sinks);
}

// Which of the 32 keys from `key` on it attends.
__device__ __forceinline__ uint32_t window_bits(const TreeParams& P, int p, int key) {
  const auto below = [](int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1; };  // the first n
  const int ahead = p - key;  // (ahead - window would leave 32 bits)
  return below(ahead + 1) & (~(ahead >= P.window ? below(ahead - P.window + 1) : 0u) | below(P.sinks - key));
}

// Adds to one row's result what was taken out of its product: the non-finite elements of the
// values that it attends and another row of its tile does not. The row's token stands at p. The
// result is fp16 (`out`) or an fp32 partial one
// (`part`, `stride` apart); dims d0, d0 + step, ... below d1. Rare, hence not inlined.
template <bool Q8, int UNIT, int CHUNK>
__device__ __noinline__ void window_patch(const TreeParams& P, const WindowTile& t, int p, __half* out, float* part,
                                          int stride, int d0, int step, int d1) {
  const int32_t* table = P.block_tables + int64_t(t.b) * P.max_blocks_per_seq;
  const int p0 = t.first();
  for (int part_of = 0; part_of < 2; ++part_of) {
    const int from = part_of ? p0 + 1 : max(t.lo, P.sinks), upto = part_of ? t.L : min(t.lo1, p0 + 1);
    for (int key = from; key < upto; ++key) {
      const int c = key / CHUNK, s = (c < t.far ? c : c - t.skip) / (UNIT / CHUNK);
      if (s < t.s0 || s >= t.s1 || !window_sees(P, p, key)) continue;
      const int block = table[key / P.block_size];
      if (block < 0 || block >= P.num_blocks) continue;
      const int64_t row = ((int64_t(block) * P.block_size + key % P.block_size) * P.kv_heads + t.kvh) * P.hv;
      for (int d = d0; d < d1; d += step) {
        const float v = Q8 ? h2f2(e4m3x2_half2(P.value_cache[row + d])).x
                           : __half2float(*reinterpret_cast<const __half*>(P.value_cache + 2 * (row + d)));
        if (isfinite(v)) continue;
        if (out) out[d] = __float2half_rn(__half2float(out[d]) + v);
        else part[int64_t(d) * stride] += v;
      }
    }
  }
}

template <int UNIT, int NR, int LEAD>
struct WindowLine {
  int tt, parts;  // whole tokens of a tile, parts of a token's heads

  __host__ __device__ __forceinline__ explicit WindowLine(const TreeSplit& S) : tt(S.tile_tokens), parts(S.tile_parts) {}

  // Sequence b's tokens, and the tiles that they make for a kv head. The tokens count as stated (at
  // most all that there are) whether the lengths keep the constraints or not.
  struct Seq {
    int q, L, tiles;  // token tiles; 0: none
  };

  // The keys between the sinks and the window of a token at position p.
  static __host__ __device__ __forceinline__ int64_t left_out(const TreeParams& P, int64_t p) {
    const int64_t n = p + 1 - P.window - P.sinks;
    return n > 0 ? n : 0;
  }

  // The places of the first t of a sequence's tiles.
  __host__ __device__ __forceinline__ int64_t upto(const TreeParams& P, const Seq& s, int t) const {
    if (t == 0) return 0;
    if (s.tiles == 1) return s.L - left_out(P, s.L - s.q) + LEAD * UNIT;
    const int64_t n = t, pre = s.L - s.q, c = pre + 1 - P.window - P.sinks;
    int64_t sum = n * (pre + LEAD * UNIT) + tt * (n * (n + 1) / 2);
    if (t == s.tiles) sum -= n * tt - s.q;
    const int64_t from = c > 0 ? 0 : tree_div(-c, tt) + 1;  // the first tile that leaves keys out
    if (n > from) sum -= (n - from) * c + tt * ((n * (n - 1) - from * (from - 1)) / 2);
    return sum;
  }

  __host__ __device__ __forceinline__ Seq load(const TreeParams& P, int b) const {
    if (b >= P.batch) return Seq{0, 0, 0};
    Seq s;
    s.q = P.q_seqlens ? P.q_seqlens[b] : 1;
    s.L = P.context_lens[b];
    const bool ok = tree_lengths_ok(P, s.q, s.L);
    if (!ok && !tree_padding(P, s.L)) tree_bad_length(P);
    s.q = tree_tokens(P, 0, max(s.q, 0));
    s.tiles = !ok || s.q == 0 ? 0 : s.q <= tt ? 1 : (s.q - 1) / tt + 1;
    return s;
  }
  // Places of all parts of all kv heads.
  __host__ __device__ __forceinline__ int64_t total(const TreeParams& P, const Seq& s) const {
    return upto(P, s, s.tiles) * (P.kv_heads * parts);
  }

  // The last worker whose piece begins before place u: total * k / n < u. (The product leaves 64 bits
  // for thousands of sequences of 2^30 keys only.)
  static __host__ __device__ __forceinline__ int last_before(int64_t total, int64_t u, int n) {
    const int64_t k = u < (int64_t(1) << 44) ? tree_div(u * n - 1, total)
                                             : int64_t((static_cast<unsigned __int128>(u) * n - 1) / total);
    return min(int(k), n - 1);
  }
};

// One worker's way along the line (warp-collective, every lane the same). It finds its first tile by the
// sums and goes on from tile to tile.
template <int UNIT, int CHUNK, int NR, int LEAD>
struct WindowWalk {
  using Line = WindowLine<UNIT, NR, LEAD>;
  int64_t u, u0, u1, total;
  int64_t at;        // the place where the tile at hand begins,
  int head, tile;    // part of a kv head's heads, token tile
  int q_start, b, nact, worker;
  typename Line::Seq seq;

  // The worker's piece of a line of `total` places; none for a worker that is not needed.
  __host__ __device__ __forceinline__ bool share(const TreeSplit& S) {
    nact = total >= int64_t(S.workers) * S.min_units ? S.workers : max(int(tree_div(total, S.min_units)), 1);
    if (worker >= nact) return false;
    // piece c begins at total * c / nact
    const int64_t each = tree_div(total, nact), rest = total - each * nact;
    u = u0 = each * worker + tree_div(rest * worker, nact);
    u1 = each * (worker + 1) + tree_div(rest * (worker + 1), nact);
    return true;
  }

  // The tile of the sequence at hand, which begins at place `before`, that place u0 belongs to: the last one that
  // begins at or before it.
  __host__ __device__ __forceinline__ void enter(const TreeParams& P, const Line& line, int64_t before) {
    const int64_t of_head = line.upto(P, seq, seq.tiles);
    head = int(tree_div(u0 - before, of_head));
    at = before + head * of_head;
    int end = seq.tiles;
    while (end - tile > 1) {
      const int mid = (tile + end) >> 1;
      if (line.upto(P, seq, mid) <= u0 - at) tile = mid; else end = mid;
    }
    at += line.upto(P, seq, tile);
  }

  __device__ __forceinline__ bool begin(const TreeParams& P, const TreeSplit& S, int w, int lane) {
    constexpr unsigned FULL = 0xffffffffu;
    worker = w;
    u = u0 = u1 = at = 0;
    head = tile = q_start = 0;
    b = -1;
    const Line line(S);
    // places and tokens of 32 sequences up to this lane's (the tokens stop at all that there are)
    int64_t places;
    int tokens;
    const auto scan = [&] {
      places = line.total(P, seq);
      tokens = seq.q;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(FULL, places, o);
        const int ut = __shfl_up_sync(FULL, tokens, o);
        if (lane >= o) {
          places += up;
          tokens = tree_tokens(P, tokens, ut);
        }
      }
    };
    seq = line.load(P, lane);
    scan();
    total = __shfl_sync(FULL, places, 31);
    if (P.batch > 32) {
      int64_t rest = 0;
      for (int k = lane + 32; k < P.batch; k += 32) rest += line.total(P, line.load(P, k));
#pragma unroll
      for (int o = 16; o; o >>= 1) rest += __shfl_xor_sync(FULL, rest, o);
      total += rest;
    }
    if (!share(S)) return false;
    // the sequence that place u0 belongs to
    int64_t before = 0;
    for (int b0 = 0; b0 < P.batch && u0 < u1; b0 += 32) {
      if (b0) {
        seq = line.load(P, b0 + lane);
        scan();
      }
      const unsigned who = __ballot_sync(FULL, u0 - before < places);
      if (who) {
        const int l = __ffs(who) - 1;
        b = b0 + l;
        before += __shfl_sync(FULL, places - line.total(P, seq), l);
        const int ahead = __shfl_sync(FULL, tokens, l > 0 ? l - 1 : 0);
        if (l > 0) q_start = tree_tokens(P, q_start, ahead);
        seq.q = __shfl_sync(FULL, seq.q, l);
        seq.L = __shfl_sync(FULL, seq.L, l);
        seq.tiles = __shfl_sync(FULL, seq.tiles, l);
        enter(P, line, before);
        return true;
      }
      before += __shfl_sync(FULL, places, 31);
      q_start = tree_tokens(P, q_start, __shfl_sync(FULL, tokens, 31));
    }
    u = u1;
    return false;
  }

  __host__ __device__ __forceinline__ bool next(const TreeParams& P, const TreeSplit& S, WindowTile& w) {
    const Line line(S);
    const int tt = line.tt, parts = line.parts;
    while (u < u1) {
      // the tile's tokens, places and units
      const int pre = seq.L - seq.q, i0 = tile * tt, i1 = min(i0 + tt, seq.q) - 1;
      const int keys = pre + i1 + 1 - int(Line::left_out(P, int64_t(pre) + i0)), width = keys + LEAD * UNIT;
      const int p0 = int(u - at), p1 = int(min(int64_t(width), p0 + (u1 - u)));
      const bool first = u == u0;
      const int64_t end = at + width;
      u += p1 - p0;
      w.lo = max(pre + i0 - P.window + 1, 0);
      w.lo1 = max(pre + i1 - P.window + 1, 0);
      const int near = w.lo / CHUNK, last = (pre + i1) / CHUNK;
      w.far = P.sinks == 0 ? 0 : min((P.sinks - 1) / CHUNK + 1, near);
      w.skip = near - w.far;
      const int units = (last - w.skip) / (UNIT / CHUNK) + 1;
      const auto cut = [&](int x) {
        return x <= LEAD * UNIT ? 0 : x == width ? units : int(tree_div(int64_t(x - LEAD * UNIT) * units, keys));
      };
      w.s0 = cut(p0);
      w.s1 = cut(p1);
      w.b = b;
      w.q_start = q_start;
      w.q = i1 + 1;
      w.L = pre + i1 + 1;
      w.kvh = parts == 1 ? head : head / parts;
      w.r0 = i0 * P.group + (head - w.kvh * parts) * NR;
      w.token0 = i0;
      const bool missing = tree_rows_missing(P, q_start, seq.q);
      if (u == end) {  // on to the next tile
        at = end;
        if (++tile == seq.tiles) {
          tile = 0;
          if (++head == P.kv_heads * parts && u < u1) {
            head = 0;
            do {
              q_start = tree_tokens(P, q_start, seq.q);
              if (++b >= P.batch) {  // only if the lengths changed under the kernel
                u = u1;
                break;
              }
              seq = line.load(P, b);
            } while (seq.tiles == 0);
          }
        }
      }
      if (w.s0 == w.s1) continue;  // nothing but a lead, or less than a unit: the next worker's
      if (missing) tree_bad_length(P);
      w.slot = w.s0 == 0 && w.s1 == units ? -1 : 2 * worker + (first ? 0 : 1);
      w.parts = 0;
      if (w.s0 == 0 && w.s1 < units) w.parts = Line::last_before(total, end, nact) - worker + 1;
      return true;
    }
    return false;
  }
};

}  // namespace pa
