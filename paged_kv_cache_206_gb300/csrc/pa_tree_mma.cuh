// Tree attention on the warp-level tensor instructions, for up to 16 rows (a
// group of heads times a few drafts) per tile and K and V heads of up to 64, 128 or 256
// dims (the copies fill what a head is short of that with zeros, which add nothing to
// a score; such dims of the output are not written), over the fp16 or the 8-bit cache.
//
// A warp takes SUB keys at a time, with the keys on the M side of m16n8k16:
//   S^T[16 keys x 8 rows] = K . Q^T        online softmax in base 2
//   O^T[16 dims x 8 rows] += V^T . P^T     fp32 accumulators in registers
// Both contractions may take their index in any order as long as the two
// operands agree, so the fragments are read with 16-byte loads of whole
// chunks of a K or V row and never shuffled: in K . Q^T lane (g, c) holds dims
// of the chunks 2c, 2c + 1, ... of key rows g and g + 8 (Q is laid out to
// match); in V^T . P^T it holds, for its keys 2c, 2c + 1, 2c + 8, 2c + 9, the chunk g
// of the row, whose element pairs become rows g and g + 8 of successive m-tiles.
// e4m3 codes are widened to fp16 on the way (exact); the XOR of the chunk index
// with the row makes both reads free of bank conflicts (2-way at 64 dims of 8
// bits, where a row is half a line).
//
// The row exponents of the 8-bit cache cost no work on the elements: K's, with
// the scale, multiply the score, and V's is added to the score's base-2
// exponent, w = 2^(x + ev - M), the sum taking w 2^-ev. Powers of two: exact. The
// weights w are rounded to fp16 (2^-11 each) for the product; sums, maxima and
// accumulators are fp32.
//
// Keys that a row does not see get weight 0; as 0 * NaN is not 0, a tile that
// reaches the drafts takes the non-finite elements out of its V rows, and adds
// them at the end to the rows that do see them.
//
// Every warp is a worker of its own (pa_tree_split.cuh): it streams the keys of
// its piece of the line through a ring of its own with TMA, from one tile into the
// next without a pause, and keeps its rows' state in registers until a tile ends. There
// is no block-wide barrier. (Copied with cp.async, 16 bytes a lane, the 64 decode steps below took
// 57 us in 8 bits and the copies alone 47; with TMA they take 50. With a CTA as the worker, its four warps taking
// turns at a tile's keys and merging in shared memory, the SMs stood idle 42 % of the
// time at 64 decode steps of 1 to 4096 tokens: every tile end drained four rings.)
#pragma once

#include "pa_decode_mma.cuh"
#include "pa_tree_split.cuh"

namespace pa {

template <int HD, bool Q8, int NT>
struct TreeMma {
  static constexpr int kWarps = 4;
  static constexpr int kRowBytes = HD * (Q8 ? 1 : 2);
  static constexpr int kChunks = kRowBytes / 16;  // 16-byte chunks of a row
  static constexpr int kElems = Q8 ? 16 : 8;      // elements of a chunk
  // keys a warp takes at a time, 4 KB of K (16 rows over 8 bits of 128 dims: 60 us with 32, 77 with 16)
  static constexpr int kSub = kRowBytes <= 128 ? 32 : 16;
  static constexpr int kMT = kSub / 16;
  static constexpr int kRows = 8 * NT;
  // what a tile costs besides its keys, in units; measured, 64 sequences of up to 4096 keys and one
  // of 4096 (8 rows of 128 dims, 8 bits): 54.4 and 15.2 us at 3, 55.3 and 15.8 at 2, 54.8 and 17.2 at 5;
  // 16 rows: 60 us at 3, 59 at 4 and 58 at 6, but 22, 23 and 25 us for 8 sequences of 2048
  static constexpr int kLead = NT == 1 ? 3 : 4;
  static constexpr uint32_t kV = kSub * kRowBytes;  // V behind K in a stage
  static constexpr uint32_t kStage = 2 * kV;
  static_assert(kV % 1024 == 0, "swizzled boxes begin on 1024 bytes");
  // CTAs of an SM (3 for tiles of 8 rows, which registers and shared memory would allow, measured the same)
  static constexpr int kCtas = kStage > 9000 ? 1 : 2;
  // a warp's shared memory: the ring, query fragments (tiles of 8 rows keep theirs in
  // registers), what the rows see, the parents, the tiles ahead, the exponents, barriers
  static constexpr uint32_t kBudget = ((227 * 1024 - 2048 * kCtas) / kCtas / kWarps) & ~1023u;
  static constexpr int kTiles = 8, kMaxStages = 5;
  static constexpr uint32_t q_off = 0;  // from the ring's end on
  static constexpr uint32_t mask_off = q_off + (NT > 1 ? kRows * HD * 2 : 0);
  static constexpr uint32_t par_off = mask_off + kRows * kTreeWords * 4;
  static constexpr uint32_t bad_off = par_off + PA_TREE_MAX_TOKENS;
  static constexpr uint32_t tile_off = bad_off + kTreeWords * 4;
  using Place = TreePlace<TreeWalk<kSub, kRows, kLead>>;
  static constexpr uint32_t place_off = (tile_off + kTiles * sizeof(TreeTile) + 7) & ~7u;
  static constexpr uint32_t exps_off = (place_off + sizeof(Place) + 15) & ~15u;  // [stage][K, V][32]
  static constexpr uint32_t bars_off = exps_off + (Q8 ? kMaxStages * 64 : 0);
  static constexpr uint32_t kRest = bars_off + kMaxStages * 8;
  static constexpr int kFit = int((kBudget - kRest) / kStage);
  static constexpr int kStages = kFit < kMaxStages ? kFit : kMaxStages;
  static_assert(kStages >= 2 && kStages + 2 <= kTiles, "ring");
  static constexpr uint32_t warp_bytes = (kStages * kStage + kRest + 1023) & ~1023u;
  static constexpr uint32_t bytes = kWarps * warp_bytes + 1024;
  static_assert((bytes + 1024) * kCtas <= 228 * 1024, "shared memory");
};

// Byte of chunk `chunk` of row `row` in a K or V stage, as the copies leave it: 128-byte
// parts of the rows, [part][row][128 bytes], or rows of 64 bytes, the chunk XORed with
// the row (the copies' swizzle), which spreads equal chunks of 8 rows over all banks.
template <int CHUNKS, int SUB>
__device__ __forceinline__ uint32_t tree_at(int chunk, int row) {
  return CHUNKS >= 8 ? (chunk >> 3) * (SUB * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4)
                     : row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4);
}

// Untiled copy of global memory into shared memory, completing on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Bounded wait of the whole warp for a phase of `bar`. Every lane polls, and the
// loop's branch goes by a vote, so the warp stays converged: with one lane polling
// for the others the compiler let that lane run apart from them for long after
// the wait, and every shuffle of the code behind it took some 300 cycles (a tile of
// codes 11,000 to convert instead of 2,000).
__device__ __forceinline__ bool tree_wait(uint64_t* bar, uint32_t parity, uint32_t limit = kTreeWaitLimit) {
  const uint32_t t0 = clock();
#pragma unroll 1
  do {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  } while (__all_sync(0xffffffffu, uint32_t(clock()) - t0 <= limit));
  return false;
}

// The same for a copy of the warp's own under a lowered limit (tests): its polls do not suspend, so
// that the limit decides. Not inlined: no other call reaches it.
inline __device__ __noinline__ bool tree_wait_lowered(uint64_t* bar, uint32_t parity, uint32_t limit) {
  const uint32_t t0 = clock();
#pragma unroll 1
  do {
    if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
  } while (__all_sync(0xffffffffu, uint32_t(clock()) - t0 <= limit));
  return false;
}

__device__ __forceinline__ uint4 lds128(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }

// Zeroes the non-finite elements of a word of a V row; whether there were any.
template <bool Q8>
__device__ __forceinline__ bool clear_nonfinite(uint32_t& w) {
  uint32_t hit = 0;
  if constexpr (Q8) {
#pragma unroll
    for (int k = 0; k < 32; k += 8)
      if ((w >> k & 0x7fu) == 0x7fu) hit |= 0xffu << k;
  } else {
    if ((w & 0x7c00u) == 0x7c00u) hit |= 0xffffu;
    if ((w & 0x7c000000u) == 0x7c000000u) hit |= 0xffff0000u;
  }
  w &= ~hit;
  return hit != 0;
}

template <int HD, bool Q8, int NT>
__global__ void __launch_bounds__(128, (TreeMma<HD, Q8, NT>::kCtas))
    tree_mma_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                    const __grid_constant__ TreeParams P, const __grid_constant__ TreeSplit S, int box) {
  using Cfg = TreeMma<HD, Q8, NT>;
  constexpr int SUB = Cfg::kSub, MT = Cfg::kMT, NR = Cfg::kRows;
  constexpr int RB = Cfg::kRowBytes, C = Cfg::kChunks, E = Cfg::kElems;
  constexpr int RPB = RB < 128 ? RB : 128;  // bytes of a row that lie together
  constexpr int OT = HD / 16;  // m-tiles of O^T, k-steps of S^T
  constexpr unsigned FULL = 0xffffffffu;
  extern __shared__ uint8_t smem_all[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, c = lane & 3;
  uint8_t* ring = smem_all + (-smem_u32(smem_all) & 1023u) + warp * Cfg::warp_bytes;
  uint8_t* smem = ring + Cfg::kStages * Cfg::kStage;
  uint8_t* q_s = smem + Cfg::q_off;
  uint32_t* mask_s = reinterpret_cast<uint32_t*>(smem + Cfg::mask_off);
  uint8_t* par_s = smem + Cfg::par_off;
  uint32_t* bad_s = reinterpret_cast<uint32_t*>(smem + Cfg::bad_off);
  TreeTile* tile_s = reinterpret_cast<TreeTile*>(smem + Cfg::tile_off);
  uint8_t* exps_s = smem + Cfg::exps_off;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Cfg::bars_off);  // [stage] landed
  const int worker = blockIdx.x * Cfg::kWarps + warp;

  const int G = P.group, bs = P.block_size;

  // ---- the stream of units: where it stands on the line, and in its tile
  typename Cfg::Place* place = reinterpret_cast<typename Cfg::Place*>(smem + Cfg::place_off);
  int made = 0;                             // tiles left for the arithmetic so far
  if (lane == 0) {
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
    S.join[worker].parts = 0;  // no divided tile yet
    for (int k = 0; k < Cfg::kStages; ++k) mbar_init(&full[k], 1);
    fence_barrier_init();
  }
  __syncwarp();
  if (!tree_begin(P, S, place, worker, lane)) return;
  int unit = 0, unit_end = 0, win0 = 0, cut_L = 0, cut_b = 0, cut_kvh = 0;
  // Lane l holds the places of 16 keys each that the units to come need: MT a
  // unit, 32 / MT units a window, and the next window's.
  constexpr int WIN = 32 / MT;
  int block = 0, in_block = 0, next_block = 0, next_in = 0;
  auto next_tile = [&]() {
    if (!tree_next(P, place)) return false;
    const TreeTile& t = place->tile;
    if (lane == 0) {
      tile_s[made % Cfg::kTiles] = t;
      if (t.parts) tree_note(S, worker, t);
    }
    ++made;
    cut_L = t.L;
    cut_b = t.b;
    cut_kvh = t.kvh;
    unit = t.s0;
    unit_end = t.s1;
    return true;
  };
  // The next unit's copies: boxes of `box` keys, which lie in one block. Rows behind the
  // context come with the last box and are dealt with where the drafts are.
  const uint64_t pol = policy_evict_first();
  int issued = 0, to = 0;  // units so far, the next one's stage
  auto issue = [&]() {
    if (unit >= unit_end && !next_tile()) return;
    const bool fresh = unit == place->tile.s0;
    if (fresh || unit >= win0 + WIN) {
      win0 = fresh ? unit : win0 + WIN;
#pragma unroll 1
      for (int k = fresh ? 0 : 1; k < 2; ++k) {
        block = next_block;
        in_block = next_in;
        const int at = win0 + k * WIN + lane / MT, key = at * SUB + (lane % MT) * 16, page = key / bs;
        next_in = key - page * bs;
        next_block = at < unit_end && key < cut_L ? P.block_tables[int64_t(cut_b) * P.max_blocks_per_seq + page] : 0;
      }
    }
    int blk[MT], in_blk[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      blk[m] = __shfl_sync(FULL, block, (unit - win0) * MT + m);
      in_blk[m] = __shfl_sync(FULL, in_block, (unit - win0) * MT + m);
    }
    if (lane == 0) {
      bool go[MT];
      uint32_t n = 0;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const bool there = blk[m] >= 0 && blk[m] < P.num_blocks, mine = m * 16 % box == 0 && unit * SUB + m * 16 < cut_L;
        if (!there) set_status(P.status, PA_STATUS_BIT_BLOCK_INDEX);
        go[m] = there && mine;
        n += go[m] ? 1 : 0;
      }
      if (n) mbar_arrive_expect_tx(&full[to], n * box * (2 * RB + (Q8 ? 2 : 0)));
      else mbar_arrive(&full[to]);
      uint8_t* dst = ring + to * Cfg::kStage;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (!go[m]) continue;
        const int row = blk[m] * bs + in_blk[m];
#pragma unroll
        for (int part = 0; part < (RB + 127) / 128; ++part) {
          uint8_t* at = dst + part * SUB * 128 + m * 16 * RPB;
          tma_load_3d(at, &tmk, &full[to], part * 128, cut_kvh, row, pol);
          tma_load_3d(at + Cfg::kV, &tmv, &full[to], part * 128, cut_kvh, row, pol);
        }
        if constexpr (Q8) {
          const int64_t e = (int64_t(blk[m]) * P.kv_heads + cut_kvh) * bs + in_blk[m];
          bulk_load(exps_s + to * 64 + m * 16, P.key_exps + e, box, &full[to]);
          bulk_load(exps_s + to * 64 + 32 + m * 16, P.value_exps + e, box, &full[to]);
        }
      }
    }
    __syncwarp();
    ++unit;
    ++issued;
    if (++to == Cfg::kStages) to = 0;
  };
#pragma unroll 1
  for (int n = 0; n < Cfg::kStages; ++n) issue();

  int n = 0, stage = 0, phase = 0;  // units done, the next one's stage
  for (int done = 0; done < made; ++done) {
    __syncwarp();
    const TreeTile t = tile_s[done % Cfg::kTiles];
    const int L = t.L, prefix = L - t.q;
    const bool drafts = t.s1 * SUB > prefix;  // the keys reach the current tokens

    // ---- the query rows as B fragments: dims of the chunks 2c, 2c + 1, ...
    uint2 qf[NT == 1 ? OT : 1];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = t.r0 + nt * 8 + g, i = r / G;
      const int64_t tok = int64_t(t.q_start) + i;
      const bool in = i < t.q && tok < P.tokens;
      const __half* src = P.query + (in ? (tok * P.num_heads + t.kvh * G + r % G) * P.hk : 0);
#pragma unroll
      for (int ks = 0; ks < OT; ++ks) {
        const int s = ks / (E / 4), j = ks % (E / 4);
        const int ch = C >= 8 ? 2 * c + (s & 1) + 8 * (s >> 1) : c;
        const bool some = in && ch * E + 4 * j < P.hk;
          const uint2 v = some ? *reinterpret_cast<const uint2*>(src + ch * E + 4 * j) : make_uint2(0, 0);
        if constexpr (NT == 1) qf[ks] = v;
        else *reinterpret_cast<uint2*>(q_s + ((nt * OT + ks) * 32 + lane) * 8) = v;
      }
    }
    // ---- what the rows see of the drafts
    if (drafts) {
      if (lane < kTreeWords) bad_s[lane] = 0;
      if (P.parents) {
        // parents as bytes (255: a root), then every row's walk to its root
        for (int i = lane; i < t.q; i += 32) {
          const int up = int64_t(t.q_start) + i < P.tokens ? P.parents[t.q_start + i] : -1;
          const bool ok = up >= -1 && up < i;
          if (!ok) set_status(P.status, PA_STATUS_BIT_TREE);
          par_s[i] = ok && up >= 0 ? uint8_t(up) : 255;
        }
        __syncwarp();
        if (lane < NR) {
          uint32_t* bits = mask_s + lane * kTreeWords;
#pragma unroll
          for (int w = 0; w < kTreeWords; ++w) bits[w] = 0;
          for (int i = (t.r0 + lane) / G; i < t.q; i = par_s[i]) {
            bits[i >> 5] |= 1u << (i & 31);
            if (par_s[i] == 255) break;
          }
        }
      }
      __syncwarp();
    }
    auto sees = [&](int row, int a) {  // draft a from a row of the tile
      return P.parents ? (mask_s[row * kTreeWords + (a >> 5)] >> (a & 31) & 1u) != 0
                       : a <= (t.r0 + row) / G;
    };

    float m_run[NT][2], l_run[NT][2], o[OT][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m_run[nt][0] = m_run[nt][1] = -INFINITY;
      l_run[nt][0] = l_run[nt][1] = 0.f;
#pragma unroll
      for (int k = 0; k < OT; ++k) o[k][nt][0] = o[k][nt][1] = o[k][nt][2] = o[k][nt][3] = 0.f;
    }

    for (int un = t.s0; un < t.s1; ++un, ++n) {
      if (!(P.wait_limit == kTreeWaitLimit ? tree_wait(&full[stage], phase)
                                             : tree_wait_lowered(&full[stage], phase, P.wait_limit))) {
        // the copies in flight, this one among them, land before the CTA's memory is given back
        if (lane == 0) set_status(P.status, PA_STATUS_BIT_TIMEOUT);
        for (; n < issued; ++n) {
          tree_wait(&full[stage], phase);
          if (++stage == Cfg::kStages) stage = 0, phase ^= 1;
        }
        return;
      }
      uint8_t* kb = ring + stage * Cfg::kStage;
      uint8_t* vb = kb + Cfg::kV;
      const uint8_t* ex = exps_s + stage * 64;
      if (++stage == Cfg::kStages) stage = 0, phase ^= 1;
      const int j0 = un * SUB;
      const bool edge = j0 + SUB > prefix;

      // ---- S^T = K . Q^T
      float s[MT][NT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.f;
#pragma unroll
      for (int sc = 0; sc < C / 4; ++sc) {
        const uint8_t* kc = kb + tree_at<C, SUB>(C >= 8 ? 2 * c + (sc & 1) + 8 * (sc >> 1) : c, g);
        uint4 xa[MT], xb[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          xa[mt] = lds128(kc + mt * 16 * RPB);
          xb[mt] = lds128(kc + (mt * 16 + 8) * RPB);
        }
#pragma unroll
        for (int j = 0; j < E / 4; ++j) {
          const int ks = sc * (E / 4) + j;
          uint32_t a[MT][4];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            const uint32_t* wa = reinterpret_cast<const uint32_t*>(&xa[mt]);
            const uint32_t* wb = reinterpret_cast<const uint32_t*>(&xb[mt]);
            if constexpr (Q8) {
              a[mt][0] = e4m3x2_half2(wa[j]);
              a[mt][1] = e4m3x2_half2(wb[j]);
              a[mt][2] = e4m3x2_half2(wa[j] >> 16);
              a[mt][3] = e4m3x2_half2(wb[j] >> 16);
            } else {
              a[mt][0] = wa[2 * j];
              a[mt][1] = wb[2 * j];
              a[mt][2] = wa[2 * j + 1];
              a[mt][3] = wb[2 * j + 1];
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            uint2 q;
            if constexpr (NT == 1) q = qf[ks];
            else q = *reinterpret_cast<const uint2*>(q_s + ((nt * OT + ks) * 32 + lane) * 8);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) mma_16816(s[mt][nt], a[mt], q.x, q.y);
          }
        }
      }

      // ---- online softmax; s[mt][nt]: keys g, g, g + 8, g + 8, rows 2c, 2c + 1, ...
      float unscale[MT][2];  // 2^-ev of this lane's keys
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const int kk = mt * 16 + hf * 8 + g, key = j0 + kk;
          float f = P.scale_log2, add = 0.f;
          unscale[mt][hf] = 1.f;
          if constexpr (Q8) {
            int ke = ex[kk], ve = max(int(ex[32 + kk]), kExpLeastByte);
            if (edge && key >= L) ke = ve = kExpBias;  // exponents behind the context: anything
            f *= pow2(ke - kExpBias);
            add = float(ve - kExpBias);
            unscale[mt][hf] = pow2(kExpBias - ve);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float& x = s[mt][nt][2 * hf + e];
              x = fmaf(x, f, add);
            }
        }
      if (edge) {
        uint32_t seen = 0;
#pragma unroll 1
        for (int k = 0; k < MT * NT * 4; ++k) {  // score k % 4 of s[k / 4 / NT][k / 4 % NT]
          const int key = j0 + k / 4 / NT * 16 + (k >> 1 & 1) * 8 + g, row = k / 4 % NT * 8 + 2 * c + (k & 1);
          if (key < prefix || (key < L && sees(row, key - prefix))) seen |= 1u << k;
        }
#pragma unroll
        for (int k = 0; k < MT * NT * 4; ++k)
          if (!(seen >> k & 1u)) s[k / 4 / NT][k / 4 % NT][k % 4] = -INFINITY;
      }
      float alpha[NT][2];
      bool moved = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(s[0][nt][e], s[0][nt][2 + e]);
#pragma unroll
          for (int mt = 1; mt < MT; ++mt) mx = fmaxf(mx, fmaxf(s[mt][nt][e], s[mt][nt][2 + e]));
          mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 16));
          const float mn = fmaxf(m_run[nt][e], mx), ref = mn == -INFINITY ? 0.f : mn;
          alpha[nt][e] = ex2(m_run[nt][e] - ref);
          moved |= mn != m_run[nt][e];
          m_run[nt][e] = mn;
          float sum = 0.f;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
              float& x = s[mt][nt][2 * hf + e];
              x = ex2(x - ref);
              sum = Q8 ? fmaf(x, unscale[mt][hf], sum) : sum + x;
            }
          l_run[nt][e] = fmaf(l_run[nt][e], alpha[nt][e], sum);
        }
      if (__any_sync(FULL, moved)) {
#pragma unroll
        for (int k = 0; k < OT; ++k)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            o[k][nt][0] *= alpha[nt][0];
            o[k][nt][1] *= alpha[nt][1];
            o[k][nt][2] *= alpha[nt][0];
            o[k][nt][3] *= alpha[nt][1];
          }
      }
      if (edge) {
        // V rows behind the context hold anything and become 0, and non-finite elements of
        // the drafts' leave the product
#pragma unroll 1
        for (int at = lane; at < SUB * C; at += 32) {
          const int row = at / C, key = j0 + row;
          if (key < prefix) continue;
          uint4* p = reinterpret_cast<uint4*>(vb + tree_at<C, SUB>(at % C, row));
          if (key >= L) {
            *p = make_uint4(0, 0, 0, 0);
            continue;
          }
          uint4 v = *p;
          bool hit = clear_nonfinite<Q8>(v.x);
          hit |= clear_nonfinite<Q8>(v.y);
          hit |= clear_nonfinite<Q8>(v.z);
          hit |= clear_nonfinite<Q8>(v.w);
          if (hit) {
            *p = v;
            const int a = key - prefix;
            atomicOr(&bad_s[(a >> 5) % kTreeWords], 1u << (a & 31));
          }
        }
        __syncwarp();
      }

      // ---- O^T += V^T . P^T
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          pb[nt][0] = movmatrix_t(pack_half2(s[mt][nt][0], s[mt][nt][1]));
          pb[nt][1] = movmatrix_t(pack_half2(s[mt][nt][2], s[mt][nt][3]));
        }
        // this lane's keys 2c, 2c + 1, 2c + 8, 2c + 9 (rows mt * 16 + ...)
        const uint8_t* v0 = vb + (mt * 16 + 2 * c) * RPB;
        if constexpr (C >= 8) {
#pragma unroll
          for (int uu = 0; uu < C / 8; ++uu) {
            const int even = uu * SUB * 128 + (g ^ (2 * c)) * 16, odd = uu * SUB * 128 + (g ^ (2 * c + 1)) * 16;
            const uint4 x0 = lds128(v0 + even), x1 = lds128(v0 + RPB + odd);
            const uint4 x2 = lds128(v0 + 8 * RPB + even), x3 = lds128(v0 + 9 * RPB + odd);
            const uint32_t *w0 = reinterpret_cast<const uint32_t*>(&x0), *w1 = reinterpret_cast<const uint32_t*>(&x1);
            const uint32_t *w2 = reinterpret_cast<const uint32_t*>(&x2), *w3 = reinterpret_cast<const uint32_t*>(&x3);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              if constexpr (Q8) {
                const uint32_t lo01 = __byte_perm(w0[j], w1[j], 0x5140), hi01 = __byte_perm(w0[j], w1[j], 0x7362);
                const uint32_t lo23 = __byte_perm(w2[j], w3[j], 0x5140), hi23 = __byte_perm(w2[j], w3[j], 0x7362);
                const uint32_t a[4] = {e4m3x2_half2(lo01), e4m3x2_half2(lo01 >> 16), e4m3x2_half2(lo23),
                                       e4m3x2_half2(lo23 >> 16)};
                const uint32_t d[4] = {e4m3x2_half2(hi01), e4m3x2_half2(hi01 >> 16), e4m3x2_half2(hi23),
                                       e4m3x2_half2(hi23 >> 16)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  mma_16816(o[uu * 8 + 2 * j][nt], a, pb[nt][0], pb[nt][1]);
                  mma_16816(o[uu * 8 + 2 * j + 1][nt], d, pb[nt][0], pb[nt][1]);
                }
              } else {
                const uint32_t a[4] = {__byte_perm(w0[j], w1[j], 0x5410), __byte_perm(w0[j], w1[j], 0x7632),
                                       __byte_perm(w2[j], w3[j], 0x5410), __byte_perm(w2[j], w3[j], 0x7632)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_16816(o[uu * 4 + j][nt], a, pb[nt][0], pb[nt][1]);
              }
            }
          }
        } else {
          // 64 dims of 8 bits: the lane's share of a row is half a chunk
          uint2 x[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int row = 2 * c + (k & 1) + 8 * (k >> 1);
            x[k] = *reinterpret_cast<const uint2*>(vb + tree_at<C, SUB>(g >> 1, mt * 16 + row) + (g & 1) * 8);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t w0 = j ? x[0].y : x[0].x, w1 = j ? x[1].y : x[1].x;
            const uint32_t w2 = j ? x[2].y : x[2].x, w3 = j ? x[3].y : x[3].x;
            const uint32_t lo01 = __byte_perm(w0, w1, 0x5140), hi01 = __byte_perm(w0, w1, 0x7362);
            const uint32_t lo23 = __byte_perm(w2, w3, 0x5140), hi23 = __byte_perm(w2, w3, 0x7362);
            const uint32_t a[4] = {e4m3x2_half2(lo01), e4m3x2_half2(lo01 >> 16), e4m3x2_half2(lo23),
                                   e4m3x2_half2(lo23 >> 16)};
            const uint32_t d[4] = {e4m3x2_half2(hi01), e4m3x2_half2(hi01 >> 16), e4m3x2_half2(hi23),
                                   e4m3x2_half2(hi23 >> 16)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma_16816(o[2 * j][nt], a, pb[nt][0], pb[nt][1]);
              mma_16816(o[2 * j + 1][nt], d, pb[nt][0], pb[nt][1]);
            }
          }
        }
      }
      // the stage's next copy comes by another proxy and waits neither for the loads nor for the
      // stores of this one by itself
      fence_proxy_async();
      __syncwarp();
      issue();
    }
    if (place->walk.u >= place->walk.u1 && done + 1 == made) launch_dependents();  // this worker's last tile

    // ---- the end of a tile
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = l_run[nt][e];
        l += __shfl_xor_sync(FULL, l, 4);
        l += __shfl_xor_sync(FULL, l, 8);
        l += __shfl_xor_sync(FULL, l, 16);
        l_run[nt][e] = l;
      }
    constexpr int DL = HD / 8;             // dims of a lane's share of a row,
    constexpr int RUN = E < DL ? E : DL;   // in runs of RUN next to one another
    constexpr int KR = RUN / 2;            // m-tiles of a run
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = nt * 8 + 2 * c + e, r = t.r0 + row, i = r / G;
        const int64_t tok = int64_t(t.q_start) + i;
        if (i >= t.q || tok >= P.tokens) continue;
        if (t.slot < 0) {
          const float inv = 1.f / l_run[nt][e];
          __half* dst = P.out + (tok * P.num_heads + t.kvh * G + r % G) * P.hv;
#pragma unroll
          for (int k0 = 0; k0 < OT; k0 += 4) {
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) h[k] = pack_half2(o[k0 + k][nt][e] * inv, o[k0 + k][nt][2 + e] * inv);
            const int d = (g + 8 * (k0 / KR)) * RUN + k0 % KR * 2;
            if (d < P.hv) *reinterpret_cast<uint4*>(dst + d) = make_uint4(h[0], h[1], h[2], h[3]);
          }
        } else {
          const int64_t at = int64_t(t.slot) * NR + row;
#pragma unroll
          for (int k = 0; k < OT; k += 2)
            *reinterpret_cast<float4*>(S.part_o + at * HD + (g + 8 * (k / KR)) * RUN + k % KR * 2) =
                make_float4(o[k][nt][e], o[k][nt][2 + e], o[k + 1][nt][e], o[k + 1][nt][2 + e]);
          if (g == 0) S.part_ml[at] = make_float2(m_run[nt][e], l_run[nt][e]);
        }
      }
    __syncwarp();
    if (drafts) {
      uint32_t hit = 0;
      for (int w = 0; w < kTreeWords; ++w) hit |= bad_s[w];
      if (hit) {
        for (int row = 0; row < NR; ++row) {
          const int r = t.r0 + row, i = r / G;
          const int64_t tok = int64_t(t.q_start) + i;
          if (i >= t.q || tok >= P.tokens) continue;
          tree_patch<Q8>(P, t.b, t.q, prefix, t.kvh, i, bad_s, P.parents ? mask_s + row * kTreeWords : nullptr,
                         t.s0 * SUB, t.s1 * SUB,
                         t.slot < 0 ? P.out + (tok * P.num_heads + t.kvh * G + r % G) * P.hv : nullptr,
                         S.part_o + (int64_t(max(t.slot, 0)) * NR + row) * HD, 1, lane, 32, P.hv);
        }
        __syncwarp();
      }
    }
  }
}

// Launches the kernel of a tile shape and its combine pass; with `need`, only
// says how much workspace they take.
cudaError_t tree_mma_64(const TreeParams& P, bool q8, int nt, int sms, size_t* need, void* ws, cudaStream_t s);
cudaError_t tree_mma_128(const TreeParams& P, bool q8, int nt, int sms, size_t* need, void* ws, cudaStream_t s);
cudaError_t tree_mma_256(const TreeParams& P, bool q8, int nt, int sms, size_t* need, void* ws, cudaStream_t s);

}  // namespace pa
