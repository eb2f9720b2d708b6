// How pa_tree_forward's warp kernels divide a batch: one line, cut into equal
// pieces.
//
// A row tile is up to NR rows of one (sequence, kv head): row r of the pair is
// token r / G, head kvh * G + r % G. Every tile walks its sequence's keys in
// units of UNIT keys, so sequence b has Hk * RT_b tiles of NU_b = ceil(L_b / UNIT)
// units. On the line a tile takes LEAD + NU_b places, in the order (b, kv head,
// row tile): LEAD stands for what a tile costs before its first and after
// its last key. Worker c of n takes the c-th n-th of the line; a place of the lead
// belongs to unit 0. A worker thus meets at most one tile that began before its
// piece, any number of whole ones, and at most one that goes on behind it; the
// two incomplete ones leave partial results (slots 2c and 2c + 1). The worker that has
// a divided tile's first keys also leaves a note of it, by which the combine kernel
// joins the parts in key order. The lengths are read on the device only, so a launch
// fits any.
//
// Where a worker has more than kSegmentKeys keys of a tile it takes them in segments of that many, each one a
// tile to the kernels, and adds up their results itself (tree_fold). The tensor cores' fp32 sums
// cut off what an addition of 16 keys rounds, always towards zero, so that their error grows with the keys: equal
// values came out 5.7e-3 too small over 2^20 keys of one worker, 5.7e-4 over 2^17. Segments are a kernel form of
// their own (SEG), chosen where the tables allow a tile of more keys: with them in every form, calls of short
// contexts took up to 4 % longer (drafts of 1024 keys 50.2 -> 51.9 us, trees of 16 94.3 -> 95.4). 2048 tokens at the end
// of 2^20 keys, 32 heads of 128 on 8, fp16, take 30.0 ms in them, 29.1 without.
#pragma once

#include "pa_tree.cuh"

namespace pa {

// A divided tile, noted by the worker that has its first keys: rows r0 .. of
// (sequence tokens q_start ..+ q, kvh), in `parts` pieces, 0 for none.
struct alignas(8) TreeJoin {
  int parts, first_slot, q_start, q, kvh, r0;
};

struct TreeSplit {
  // [2 * workers][NR][hv], not yet divided by the sum; one a worker more, for the segment at hand, where there are any
  float* part_o;
  float2* part_ml;  // the same [NR]: running maximum (base 2) and sum
  struct TreeJoin* join;  // [workers]
  int workers;
  int min_units;    // fewest places of the line worth a worker
  int tile_tokens, tile_parts;  // (pa_window_split.cuh) whole tokens of a row tile, parts of a token's heads
  float2* fold_ml;  // [2][workers][NR] of the segments so far; by halves of the columns where two threads have them
  int segment;      // units of a segment
};

// a / b for a >= 0, b > 0: the 64-bit division takes several times the 32-bit one's time.
__host__ __device__ __forceinline__ int64_t tree_div(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return uint32_t(a) / uint32_t(b);
  return a / b;
}

template <int UNIT, int NR, int LEAD>
struct TreeLine {
  // Sequence b's tokens, row tiles of a kv head and units of a tile; a sequence
  // whose lengths break a constraint has no tiles, but as many tokens as it states (at
  // most all that there are): the rows of the next one lie behind them.
  struct Seq {
    int q, L, tiles, units;
    __device__ __forceinline__ int places() const { return units + LEAD; }  // of a tile
    __device__ __forceinline__ int64_t total(const TreeParams& P) const {
      return int64_t(P.kv_heads) * tiles * places();
    }
  };
  static __device__ __forceinline__ Seq load(const TreeParams& P, int b) {
    if (b >= P.batch) return Seq{0, 0, 0, 0};
    Seq s;
    s.q = P.q_seqlens ? P.q_seqlens[b] : 1;
    s.L = P.context_lens[b];
    const bool ok = tree_lengths_ok(P, s.q, s.L);
    if (!ok && !tree_padding(P, s.L)) set_status(P.status, PA_STATUS_BIT_PLAN);
    s.q = tree_tokens(P, 0, max(s.q, 0));
    const bool some = ok && s.q > 0;
    s.tiles = some ? (s.q * P.group - 1) / NR + 1 : 0;
    s.units = some ? (s.L - 1) / UNIT + 1 : 0;
    return s;
  }

  // The places and tokens of 32 sequences up to this lane's, its own among them (the
  // tokens stop at all that there are).
  struct Sums {
    int64_t places;
    int tokens;
  };
  static __device__ __forceinline__ Sums scan(const TreeParams& P, int lane, const Seq& s) {
    Sums u{s.total(P), s.q};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, u.places, o);
      const int ut = __shfl_up_sync(0xffffffffu, u.tokens, o);
      if (lane >= o) {
        u.places += up;
        u.tokens = tree_tokens(P, u.tokens, ut);
      }
    }
    return u;
  }

  // Workers that share the line, and where worker c's piece begins.
  static __device__ __forceinline__ int active(int64_t total, int workers, int min_units) {
    const int64_t n = tree_div(total, min_units);
    return int(n < 1 ? 1 : n < workers ? n : workers);
  }
  static __device__ __forceinline__ int64_t begin(int64_t total, int c, int n) {
    return tree_div(total * c, n);
  }
  // The last worker whose piece begins before place u: total * k / n < u.
  static __device__ __forceinline__ int last_before(int64_t total, int64_t u, int n) {
    return min(int(tree_div(u * n - 1, total)), n - 1);
  }
};

// The keys of one row tile that one worker has.
struct TreeTile {
  int b, q_start, q, L, kvh, r0;
  int s0, s1;  // units [s0, s1)
  int slot;    // of a partial result; -1: the whole tile
  int parts;   // of a divided tile whose first keys are here, else 0
  static constexpr bool kSegments = false;
};

// The same of a kernel that takes segments.
template <class Tile>
struct TreeSegment : Tile {
  // Of a segment, whose slot is the worker's third: 4 * (the slot that the tile has + 2), and 1 for the first
  // one, 2 for the last one; else 0.
  int seg;
  int end;  // the tile's, where it goes on in another segment; else 0
  static constexpr bool kSegments = true;
};

// Keys of a segment. (A tile of 256 rows takes 0.9 ms for them and 4 to 10 us at its ends.)
constexpr int kSegmentKeys = 1 << 16;

// Whether a tile of this many rows may have more keys than that.
inline bool tree_segments(const TreeParams& P, int rows) {
  const int64_t seen = int64_t(P.window) + P.sinks + rows;
  return (P.window && seen < P.max_keys ? seen : P.max_keys) > kSegmentKeys;
}

// One worker's way along the line (warp-collective, every lane the same).
template <int UNIT, int NR, int LEAD>
struct TreeWalk {
  using Line = TreeLine<UNIT, NR, LEAD>;
  int64_t u, u0, u1, before, total;
  int q_start, b, nact, worker;
  typename Line::Seq seq;

  __device__ __forceinline__ bool begin(const TreeParams& P, const TreeSplit& S, int w, int lane) {
    worker = w;
    u = u0 = u1 = before = 0;
    q_start = 0;
    b = -1;
    // the line's length: of the first 32 sequences (kept for the search) and the others
    seq = Line::load(P, lane);
    typename Line::Sums sums = Line::scan(P, lane, seq);
    total = __shfl_sync(0xffffffffu, sums.places, 31);
    if (P.batch > 32) {
      int64_t rest = 0;
      for (int k = lane + 32; k < P.batch; k += 32) rest += Line::load(P, k).total(P);
#pragma unroll
      for (int o = 16; o; o >>= 1) rest += __shfl_xor_sync(0xffffffffu, rest, o);
      total += rest;
    }
    nact = Line::active(total, S.workers, S.min_units);
    if (worker >= nact) return false;
    u = u0 = Line::begin(total, worker, nact);
    u1 = Line::begin(total, worker + 1, nact);
    // the sequence that place u0 belongs to
    for (int b0 = 0; b0 < P.batch && u0 < u1; b0 += 32) {
      if (b0) {
        seq = Line::load(P, b0 + lane);
        sums = Line::scan(P, lane, seq);
      }
      const unsigned who = __ballot_sync(0xffffffffu, u0 - before < sums.places);
      if (who) {
        const int l = __ffs(who) - 1;
        b = b0 + l;
        before += __shfl_sync(0xffffffffu, sums.places - seq.total(P), l);
        const int ahead = __shfl_sync(0xffffffffu, sums.tokens, l > 0 ? l - 1 : 0);
        if (l > 0) q_start = tree_tokens(P, q_start, ahead);
        seq.q = __shfl_sync(0xffffffffu, seq.q, l);
        seq.L = __shfl_sync(0xffffffffu, seq.L, l);
        seq.tiles = __shfl_sync(0xffffffffu, seq.tiles, l);
        seq.units = __shfl_sync(0xffffffffu, seq.units, l);
        return true;
      }
      before += __shfl_sync(0xffffffffu, sums.places, 31);
      q_start = tree_tokens(P, q_start, __shfl_sync(0xffffffffu, sums.tokens, 31));
    }
    u = u1;
    return false;
  }

  __device__ __forceinline__ bool next(const TreeParams& P, const TreeSplit&, TreeTile& t) {
    while (u < u1) {
      while (u >= before + seq.total(P)) {
        before += seq.total(P);
        q_start = tree_tokens(P, q_start, seq.q);
        if (++b >= P.batch) {  // only if the lengths changed under the kernel
          u = u1;
          return false;
        }
        seq = Line::load(P, b);
      }
      const int tile = int(tree_div(u - before, seq.places()));
      const int p0 = int(u - before - int64_t(tile) * seq.places());
      const int p1 = int(min(int64_t(seq.places()), p0 + (u1 - u)));
      const bool first = u == u0;
      u += p1 - p0;
      t.s0 = max(p0 - LEAD, 0);
      t.s1 = max(p1 - LEAD, 0);
      if (t.s0 == t.s1) continue;  // nothing but a lead: the next worker's
      if (tree_rows_missing(P, q_start, seq.q)) set_status(P.status, PA_STATUS_BIT_PLAN);
      t.b = b;
      t.q_start = q_start;
      t.q = seq.q;
      t.L = seq.L;
      t.kvh = seq.tiles == 1 ? tile : tile / seq.tiles;
      t.r0 = (tile - t.kvh * seq.tiles) * NR;
      t.slot = t.s0 == 0 && t.s1 == seq.units ? -1 : 2 * worker + (first ? 0 : 1);
      t.parts = 0;
      if (t.s0 == 0 && t.s1 < seq.units)
        t.parts = Line::last_before(total, before + int64_t(tile + 1) * seq.places(), nact) - worker + 1;
      return true;
    }
    return false;
  }
};

// A warp's place on the line, in shared memory, and its steps along it as
// functions of their own: they are rare, and inlined where they are called (with
// their divisions) they pushed the kernels' loops out of the instruction cache.
// All lanes hold and store the same values.
template <class Walk, class Tile = TreeTile>
struct TreePlace {
  Walk walk;
  Tile tile;
};

template <class Walk, class Tile>
__device__ __noinline__ bool tree_begin(const TreeParams& P, const TreeSplit& S, TreePlace<Walk, Tile>* at, int worker,
                                        int lane) {
  Walk w;
  const bool some = w.begin(P, S, worker, lane);
  at->walk = w;
  if constexpr (Tile::kSegments) at->tile.end = 0;
  __syncwarp();
  return some;
}

// The first segment of the tile at hand, or its next one.
template <class Walk, class Tile>
__device__ __noinline__ void tree_next_segment(const TreeSplit& S, TreePlace<Walk, Tile>* at) {
  Tile d = at->tile;
  if (d.end) {
    d.s0 = d.s1;
    d.seg &= ~1;
    d.parts = 0;
  } else {
    d.end = d.s1;
    d.seg = 4 * (d.slot + 2) | 1;
    d.slot = 2 * S.workers + at->walk.worker;
  }
  d.s1 = min(d.s0 + S.segment, d.end);
  if (d.s1 == d.end) {
    d.seg |= 2;
    d.end = 0;
  }
  __syncwarp();
  at->tile = d;
  __syncwarp();
}

template <class Walk, class Tile>
__device__ __noinline__ bool tree_next(const TreeParams& P, const TreeSplit& S, TreePlace<Walk, Tile>* at) {
  if constexpr (Tile::kSegments)
    if (at->tile.end) {
      tree_next_segment(S, at);
      return true;
    }
  Walk w = at->walk;
  Tile d;
  const bool some = w.next(P, S, d);
  if constexpr (Tile::kSegments) d.seg = d.end = 0;
  __syncwarp();
  if (some) at->tile = d;
  at->walk = w;
  __syncwarp();
  if constexpr (Tile::kSegments)
    if (some && d.s1 - d.s0 > S.segment) tree_next_segment(S, at);
  return some;
}

// The note of a divided tile (parts = 0: none).
template <class Tile>
__device__ __forceinline__ void tree_note(const TreeSplit& S, int worker, const Tile& t) {
  int slot = t.slot;
  if constexpr (Tile::kSegments)
    if (t.seg) slot = (t.seg >> 2) - 2;
  S.join[worker] = TreeJoin{t.parts, slot, t.q_start, t.q, t.kvh, t.r0};
}

// Adds a segment's result for one row, which lies in the worker's third slot as a partial result does (column d at
// d * stride from `at`), to the tile's segments before it: in the tile's own slot, or for a whole tile
// in the worker's second one, which its last tile takes later. With the last segment a
// whole tile's row goes to `out`. `ml` is the segment's maximum and sum. By a thread for its columns [d0, d1) of the
// row, the half-th of two at most that have the row, each with a maximum and a sum of its own, or (STEP = 32) by
// a warp. Rare, hence not inlined.
template <int HD, int NR, int STEP>
__device__ __noinline__ void tree_fold(const TreeSplit& S, int worker, int seg, int half, int row, float2 ml, int64_t at,
                                       int stride, __half* out, int d0, int d1) {
  const int to = (seg >> 2) - 2, slot = to < 0 ? 2 * worker + 1 : to;
  const bool first = seg & 1, last = seg & 2;
  float2* mine = S.fold_ml + (int64_t(half) * S.workers + worker) * NR + row;
  const float2 old = first ? make_float2(-INFINITY, 0.f) : *mine;
  if (STEP == 32) __syncwarp();  // (read by every lane before one of them writes it)
  const float top = fmaxf(old.x, ml.x), ref = top == -INFINITY ? 0.f : top;
  const float wa = ex2(old.x - ref), wb = ex2(ml.x - ref), sum = old.y * wa + ml.y * wb;
  *mine = make_float2(top, sum);
  if (last && to >= 0 && half == 0) S.part_ml[int64_t(to) * NR + row] = make_float2(top, sum);
  const float* from = S.part_o + (int64_t(2 * S.workers + worker) * HD) * NR + at;
  float* acc = S.part_o + int64_t(slot) * HD * NR + at;
  // (a sum that is no number stays so however little it weighs)
  const auto times = [](float x, float w) { return isfinite(x) ? x * w : x; };
  for (int d = d0; d < d1; d += STEP) {
    float x = times(from[int64_t(d) * stride], wb);
    if (!first) x += times(acc[int64_t(d) * stride], wa);
    if (last && to < 0) out[d] = __float2half_rn(x / sum);
    else acc[int64_t(d) * stride] = x;
  }
}

// Joins the partial results of the divided tiles: CTA (c, y) the rows [8 y, 8 y + 8)
// of the tile that worker c noted, a warp a row. Launched as the attention
// kernel's programmatic dependent. The maxima and sums of 32 parts are read by a lane each,
// and 16 parts' rows are on their way meanwhile: at 4096 keys of one decode step
// a tile has 43 parts, and they come in three waits.
template <int HD, int NR>
__global__ void __launch_bounds__(256) tree_combine_kernel(const TreeParams P, const TreeSplit S) {
  constexpr int DPL = HD / 32;  // dims a lane holds, next to one another
  constexpr int BATCH = 8;  // partial rows in flight
  const int lane = threadIdx.x & 31, n = blockIdx.y * 8 + (threadIdx.x >> 5);
  grid_dependency_wait();
  const TreeJoin t = S.join[blockIdx.x];
  if (t.parts == 0) return;
  const int r = t.r0 + n, i = r / P.group;
  const int64_t tok = int64_t(t.q_start) + i;
  if (i >= t.q || tok >= P.tokens) return;
  // part 0 is the noting worker's last tile, the others the next workers' first
  auto row_of = [&](int k) {
    return int64_t(k == 0 ? t.first_slot : 2 * (int(blockIdx.x) + k)) * NR + n;
  };
  float x[BATCH][DPL];
  auto load = [&](int k0) {
#pragma unroll
    for (int k = 0; k < BATCH; ++k)
      if (k0 + k < t.parts)
#pragma unroll
        for (int d = 0; d < DPL; d += 2)
          *reinterpret_cast<float2*>(&x[k][d]) =
              *reinterpret_cast<const float2*>(S.part_o + row_of(k0 + k) * HD + lane * DPL + d);
  };
  float M = -INFINITY, sum = 0.f, w = 0.f, acc[DPL];
#pragma unroll
  for (int k = 0; k < DPL; ++k) acc[k] = 0.f;
#pragma unroll 1
  for (int k0 = 0; k0 < t.parts; k0 += BATCH) {
    float2 ml = make_float2(-INFINITY, 0.f);
    if (k0 % 32 == 0 && k0 + lane < t.parts) ml = S.part_ml[row_of(k0 + lane)];
    load(k0);
    if (k0 % 32 == 0) {
      const float top = fmaxf(M, warp_max(ml.x));
      const float ref = top == -INFINITY ? 0.f : top;  // no score above -inf: weights of 0
      const float alpha = ex2(M - ref);
      M = top;
      w = ex2(ml.x - ref);
      sum = fmaf(sum, alpha, warp_sum(ml.y * w));
#pragma unroll
      for (int d = 0; d < DPL; ++d) acc[d] *= alpha;
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k0 % 32 + k);
      if (k0 + k < t.parts)
#pragma unroll
        for (int d = 0; d < DPL; ++d) acc[d] = fmaf(wk, x[k][d], acc[d]);
    }
  }
  if (lane * DPL >= P.hv) return;
  __half2* dst = reinterpret_cast<__half2*>(
      P.out + (tok * P.num_heads + t.kvh * P.group + r % P.group) * P.hv + lane * DPL);
  const float inv = 1.f / sum;
#pragma unroll
  for (int d = 0; d < DPL; d += 2) dst[d / 2] = __floats2half2_rn(acc[d] * inv, acc[d + 1] * inv);
}

// The same for wide row tiles, whose partial rows are stored by columns,
// [slot][HD][NR], so that a kernel with a row per thread stores whole lines: CTA (c, y)
// the rows [32 y, 32 y + 32), a lane a row, a warp HD / 8 columns.
template <int HD, int NR>
__global__ void __launch_bounds__(256) tree_combine_cols_kernel(const TreeParams P, const TreeSplit S) {
  constexpr int COLS = HD / 8;
  const int lane = threadIdx.x & 31, d0 = (threadIdx.x >> 5) * COLS, n = blockIdx.y * 32 + lane;
  grid_dependency_wait();
  const TreeJoin& t = S.join[blockIdx.x];
  const int parts = t.parts;
  if (parts == 0) return;
  const int r = t.r0 + n, i = r / P.group;
  const int64_t tok = int64_t(t.q_start) + i;
  if (i >= t.q || tok >= P.tokens) return;
  auto slot_of = [&](int k) { return int64_t(k == 0 ? t.first_slot : 2 * (int(blockIdx.x) + k)); };
  float M = -INFINITY, sum = 0.f, acc[COLS];
#pragma unroll
  for (int d = 0; d < COLS; ++d) acc[d] = 0.f;
  // several parts' loads in flight at a time: a tile of one long sequence has some twenty
  constexpr int BATCH = 2;
  for (int k0 = 0; k0 < parts; k0 += 4) {
    float m[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) m[k] = k0 + k < parts ? S.part_ml[slot_of(k0 + k) * NR + n].x : -INFINITY;
#pragma unroll
    for (int k = 0; k < 4; ++k) M = fmaxf(M, m[k]);
  }
  if (M == -INFINITY) M = 0.f;  // no score above -inf: the sum below is 0
  for (int k0 = 0; k0 < parts; k0 += BATCH) {
    float2 ml[BATCH];
    float x[BATCH][COLS];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      if (k0 + k >= parts) break;
      const int64_t slot = slot_of(k0 + k);
      ml[k] = S.part_ml[slot * NR + n];
#pragma unroll
      for (int d = 0; d < COLS; ++d) x[k][d] = S.part_o[(slot * HD + d0 + d) * NR + n];
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      if (k0 + k >= parts) break;
      const float w = ex2(ml[k].x - M);
      sum = fmaf(ml[k].y, w, sum);
#pragma unroll
      for (int d = 0; d < COLS; ++d) acc[d] = fmaf(w, x[k][d], acc[d]);
    }
  }
  const float inv = 1.f / sum;
  uint4* dst = reinterpret_cast<uint4*>(
      P.out + (tok * P.num_heads + t.kvh * P.group + r % P.group) * HD + d0);
#pragma unroll
  for (int d = 0; d < COLS; d += 8)
    dst[d / 8] = make_uint4(pack_half2(acc[d] * inv, acc[d + 1] * inv), pack_half2(acc[d + 2] * inv, acc[d + 3] * inv),
                            pack_half2(acc[d + 4] * inv, acc[d + 5] * inv), pack_half2(acc[d + 6] * inv, acc[d + 7] * inv));
}

}  // namespace pa
