// How pa_tree_forward's kernels divide a batch: one line of units, cut into
// equal pieces.
//
// A row tile is up to NR rows of one (sequence, kv head): row r of the pair is
// token r / G, head kvh * G + r % G. Every tile walks its sequence's keys in
// units of UNIT keys, so sequence b has Hk * RT_b * NU_b units (RT_b row tiles,
// NU_b = ceil(L_b / UNIT)); the units of the batch, in the order (b, kv head, row
// tile, unit), form one line, of which CTA c of n takes the c-th n-th. A CTA
// thus meets at most one tile that began before its piece, any number of whole
// ones, and at most one that goes on behind it; the two incomplete ones leave
// partial results (slots 2c and 2c + 1), which the combine kernel joins in key
// order. The lengths are read on the device only, so a launch fits any.
#pragma once

#include "pa_tree.cuh"

namespace pa {

struct TreeSplit {
  float* part_o;   // [2 * CTAs][NR][hv], not yet divided by the sum
  float2* part_ml; // [2 * CTAs][NR]: running maximum (base 2) and sum
  int min_units;   // fewest units worth a CTA
};

template <int UNIT, int NR>
struct TreeLine {
  // Sequence b's tokens, row tiles and units per tile; a sequence whose lengths
  // break a constraint has none.
  struct Seq {
    int q, L, tiles, units;
    __device__ __forceinline__ int64_t total(const TreeParams& P) const {
      return int64_t(P.kv_heads) * tiles * units;
    }
  };
  static __device__ __forceinline__ Seq load(const TreeParams& P, int b) {
    Seq s;
    s.q = P.q_seqlens ? P.q_seqlens[b] : 1;
    s.L = P.context_lens[b];
    const bool ok = tree_lengths_ok(P, s.q, s.L);
    if (!ok) set_status(P.status, PA_STATUS_BIT_PLAN);
    s.q = min(max(s.q, 0), P.max_q);
    const bool some = ok && s.q > 0;
    s.tiles = some ? (s.q * P.group + NR - 1) / NR : 0;
    s.units = some ? (s.L + UNIT - 1) / UNIT : 0;
    return s;
  }

  // Units of the whole batch (warp-collective).
  static __device__ __forceinline__ int64_t total(const TreeParams& P, int lane) {
    int64_t n = 0;
    for (int b = lane; b < P.batch; b += 32) n += load(P, b).total(P);
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    return n;
  }

  // The sequence that unit u of the line belongs to, the units and the tokens
  // before it (warp-collective; u below the total).
  static __device__ __forceinline__ int find(const TreeParams& P, int64_t u, int lane,
                                             int64_t& before, int& q_start) {
    before = 0;
    q_start = 0;
    for (int b0 = 0; b0 < P.batch; b0 += 32) {
      Seq s{0, 0, 0, 0};
      if (b0 + lane < P.batch) s = load(P, b0 + lane);
      const int64_t n = s.total(P);
      int64_t un = n;
      int tn = s.q;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t ua = __shfl_up_sync(0xffffffffu, un, o);
        const int ta = __shfl_up_sync(0xffffffffu, tn, o);
        if (lane >= o) {
          un += ua;
          tn += ta;
        }
      }
      const unsigned who = __ballot_sync(0xffffffffu, n > 0 && u < before + un);
      if (who) {
        const int l = __ffs(who) - 1;
        before += __shfl_sync(0xffffffffu, un - n, l);
        q_start += __shfl_sync(0xffffffffu, tn - s.q, l);
        return b0 + l;
      }
      before += __shfl_sync(0xffffffffu, un, 31);
      q_start += __shfl_sync(0xffffffffu, tn, 31);
    }
    return -1;
  }

  // CTAs that share the line, and where CTA c's piece begins.
  static __device__ __forceinline__ int ctas(int64_t total, int grid, int min_units) {
    const int64_t n = total / min_units;
    return int(n < 1 ? 1 : n < grid ? n : grid);
  }
  static __device__ __forceinline__ int64_t begin(int64_t total, int c, int n) { return total * c / n; }
};

// Joins the partial results of the tiles that more than one CTA worked on. CTA
// (c, y) takes the tile that piece c begins inside of, if c is the first piece
// that does, and its rows [8 y, 8 y + 8), a warp a row. Launched as the
// attention kernel's programmatic dependent.
template <int HD, int UNIT, int NR>
__global__ void __launch_bounds__(256) tree_combine_kernel(const TreeParams P, const TreeSplit S,
                                                           int grid) {
  using Line = TreeLine<UNIT, NR>;
  constexpr int DPL = HD / 32;  // dims a lane holds: lane, lane + 32, ...
  const int lane = threadIdx.x & 31, n = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int64_t total = Line::total(P, lane);
  const int nact = Line::ctas(total, grid, S.min_units);
  const int c = blockIdx.x + 1;
  if (c >= nact) return;
  const int64_t u = Line::begin(total, c, nact);
  int64_t before;
  int q_start;
  const int b = Line::find(P, u, lane, before, q_start);
  if (b < 0) return;
  const typename Line::Seq s = Line::load(P, b);
  const int g = int((u - before) / s.units);
  const int64_t g0 = before + int64_t(g) * s.units, g1 = g0 + s.units;
  if (u == g0 || Line::begin(total, c - 1, nact) > g0) return;  // not inside a tile, or not its first
  const int kvh = g / s.tiles, r = (g % s.tiles) * NR + n, i = r / P.group;
  const int64_t t = int64_t(q_start) + i;
  if (i >= s.q || t >= P.tokens) return;
  // pieces c - 1 .. last hold a part of the tile
  int last = c;
  while (last + 1 < nact && Line::begin(total, last + 1, nact) < g1) ++last;
  const int first_slot = 2 * (c - 1) + (Line::begin(total, c - 1, nact) == g0 ? 0 : 1);
  grid_dependency_wait();
  float M = -INFINITY;
  for (int k = c - 1 + lane; k <= last; k += 32)
    M = fmaxf(M, S.part_ml[int64_t(k == c - 1 ? first_slot : 2 * k) * NR + n].x);
  M = warp_max(M);
  if (M == -INFINITY) M = 0.f;  // no score above -inf: the sum below is 0
  float sum = 0.f, acc[DPL];
#pragma unroll
  for (int k = 0; k < DPL; ++k) acc[k] = 0.f;
  for (int k = c - 1; k <= last; ++k) {
    const int64_t row = int64_t(k == c - 1 ? first_slot : 2 * k) * NR + n;
    const float2 ml = S.part_ml[row];
    const float w = ex2(ml.x - M);
    sum += ml.y * w;
#pragma unroll
    for (int d = 0; d < DPL; ++d) acc[d] += w * S.part_o[row * HD + d * 32 + lane];
  }
  __half* dst = P.out + (t * P.num_heads + kvh * P.group + r % P.group) * HD;
#pragma unroll
  for (int d = 0; d < DPL; ++d) dst[d * 32 + lane] = __float2half_rn(acc[d] / sum);
}

}  // namespace pa
