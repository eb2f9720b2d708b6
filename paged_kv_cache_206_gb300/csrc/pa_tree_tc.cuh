// Tree attention, and attention with a window, on the tcgen05 tensor cores, for tiles of 128 or 256
// rows (a group of heads times many drafts, or a prompt's tokens) and heads of 64 or 128 dims, over
// the fp16 or the 8-bit cache.
//
// One persistent CTA per SM, a worker of the line (pa_tree_split.cuh) with units of
// 128 keys. Two chains of softmax and O += P V run against each other in jobs of 64
// keys: with up to 128 rows chain g takes half g of every key tile, S = Q K^T of
// two tiles being in TMEM, and the chains' states are joined at the end (QT = 1); with
// more rows each chain has a query tile of its own and takes both halves of every
// tile (QT = 2). The 64 scores of a row's job fit in a thread's registers, so they are
// read from TMEM once. S is made for 128 keys at a time: an MMA of half the width
// reads the query operand as often and took 500 cycles per 64 keys for the 64 it
// computes. (Jobs of 128 keys, the scores read twice: 4.6 us per 256 rows x 128 keys.)
//
//   warp 0       keys' copies (TMA)
//   warp 1       issues O_g += P_g V. O_g stands in TMEM columns [256 + 128 g, +HD)
//   warp 2       values' copies
//   warp 3       finds the row tiles on the line and tells them to the others; loads
//                their queries (cp.async); issues S = Q K^T into columns [128 x, +128), x
//                the key tile's parity (QT = 1) or the chain (QT = 2). A job's P (fp16)
//                overwrites the front of its 64 columns of S, where the other product
//                takes it as its A operand from TMEM. (One warp issuing both products took
//                2.7 us for a tile's 1,030 cycles of MMA: the waits of one stood before the other.)
//   warps 4-11   softmax, one row a thread: group g = chain g
//   warps 12-15  8-bit cache only: codes to fp16 operands, a warp for each of the
//                four 64-row parts (K, K, V, V) of a tile. The rows of a tile are
//                brought to the tile's largest exponent (code * 2^(e_j - e_max),
//                exact), so the softmax sees one factor for K and one exponent for
//                V per tile, as the fp16 cache's does. A row whose exponent lies
//                further below (kSpreadK, kSpreadV), as one row may be large that
//                others do not even attend, is brought down by that much only, and
//                the softmax applies the rest to the key's score and weight
//                (tree_apart), exactly, as the warp-level kernel always does.
//
// The reference maximum of a row moves only when a score passes it by 2^8; sums,
// maxima and accumulators are fp32, the weights fp16. Over the 8-bit cache the weights
// stand 2^kLift above that: a tile's exponent may be kSpreadV above that of every V row
// that a row attends, and its weights keep their 11 bits all the same. All roles walk the same
// tiles of the line; rings and barriers run on across them, so the copies of the
// next tile are under way while the last one's rows are written out. Every wait is
// bounded.
#pragma once

#include <cfloat>

#include "pa_prefill_tc.cuh"
#include "pa_tree_mma.cuh"

namespace pa {

// WIN: pa_window_forward's kernel, for drafts, prompts and parts of prompts. Its row tiles are those of
// pa_window_split.cuh, of some ten key tiles each where the window is of a thousand keys, so that what a row tile costs
// at its ends counts as much as the key tiles do (10 us beside 1.85 each in the division of the work above, 4
// beside 1.70 now: 256 rows of fp16):
//   warp 1       issues both products, each S behind the product that frees its columns
//   warp 3       finds the row tiles (one from the other: with a search in each it took 4 us a tile), and
//                fetches their queries by TMA (2.6 to 5 us by cp.async)
//   warps 4-11   leave out the keys that none of their rows sees, mask those that not all of them see, and
//                write the rows out, eight rows' 64 bytes a store
//   warps 12-15  fp16 cache: make the V rows that no row of the tile sees 0 and look for non-finite
//                elements in those that not every row sees, at both ends of the windows, before the product
//                (the 8-bit cache's widening warps do that on the way); of heads of 128 dims and 256 rows they
//                also write half of each row out
// Sinks and window share a key tile by halves of 64 keys.
// What it reaches: 18,700 tokens of prompts, window 1024, 32 heads on 8, in 310 to 317 us (0.98 PFLOP/s of the pairs that
// are attended, 49 % of the tensor pipe's time; chains of S, softmax and P V of two query tiles that wait for each
// other); 8 x 512 tokens over 8 bits, window 2048, 32 heads, in 162 us (0.76; the widening warps share the schedulers
// with the softmax, issue slots 42 % full).
template <int HD, bool Q8, int QT, bool WIN, bool SEG>
struct TreeTc {
  static constexpr int kConv = 1;  // warps that widen a 64-row part of codes
  static constexpr bool kLook = WIN && !Q8;  // there are warps that look the V tiles through,
  static constexpr bool kShare = kLook && HD == 128 && QT == 2;  // and write the second half of the rows out
  static constexpr int kThreads = Q8 ? 384 + 4 * 32 * kConv : kLook ? 512 : 384;
  static constexpr int kTok = 128;
  static constexpr int kRows = 128 * QT;
  // What a row tile costs next to its key tiles, in these, measured at 32 trees over 64 to 8192
  // keys, heads of 128: trees of 5 to 16 in 8 bits 108 us at 3, 97 at 5, 95 at 6, 96 at 8, 99 at 12; of
  // 64 in fp16 144 at 3, 135 at 4, 132 at 5, 136 at 8 (and 16 of those 75, 76, 77 and 81). With a window, whose tiles
  // end with less: prompts in fp16 317 at 2, 315 at 3, 320 at 4; parts in 8 bits 210, 198, - and 195 at 5, 197 at 6;
  // drafts in 8 bits 57 at 2 and 3, 60 at 5.
  static constexpr int kLead = WIN ? (Q8 && QT == 2 ? 5 : 3) : Q8 ? 6 : 4;
  static constexpr int kHalves = HD / 64;
  static constexpr uint32_t kHalf = 128 * 128;           // 64 dims of 128 fp16 rows
  static constexpr uint32_t kTile = kHalf * kHalves;     // a K or V tile, a query tile
  static constexpr int kKSlots = Q8 || QT == 2 ? 2 : 3;
  static constexpr int kVSlots = Q8 ? 1 : 2;
  static constexpr uint32_t kStageBytes = 64 * HD;       // 64 rows of codes
  // Stages for the codes rather than a second V operand (trees of 16, when this was chosen: 88.5 us, 92.3
  // with two V slots and 4 + 3 stages, 107 with one K slot and 7 + 8)
  static constexpr int kKStages = Q8 ? (QT == 1 ? 5 : 4) : 0, kVStages = Q8 ? (QT == 1 ? 6 : 3) : 0;
  static constexpr int kStages = kKStages + kVStages;
  // Barriers of the parts that have landed: of each part (rows 0.., rows 64..) of as many key tiles
  // as have parts in the ring, whatever stage a part is in. A barrier per stage would do for
  // an even number of stages; with an odd one a stage serves the two parts' warps in turn, and a
  // warp that asked for its turn while the other's copy was still in flight took the phase
  // before that one for its own (parts may land in either order).
  static constexpr int kKRounds = (kKStages + 1) / 2, kVRounds = (kVStages + 1) / 2;
  static constexpr int kLanded = 2 * (kKRounds + kVRounds);
  // Key tiles whose exponents, and whose largest ones, are held; row tiles whose flags
  // are. While the softmax has a key tile n before it, the products S reach n + 1, the K slots n + 3,
  // the widening warps' registers n + 4 (whose exponents they have told) and the K stages the first
  // half of n + 7 (the V ones n + 4), so a row tile or key tile eight on finds the place read.
  static constexpr int kExps = 8, kMeta = 8, kBad = 8;
  // How far below the tile's largest exponent a row is brought up to it: a code (a multiple of
  // 2^-9) times 2^-14 is still exact in fp16, and weights may stand 2^7 higher (2^(8 + 7) < 65504).
  static constexpr int kSpreadK = 14, kSpreadV = 7, kLift = Q8 ? kSpreadV : 0;
  static constexpr int kAhead = 4;                       // row tiles told to the roles
  static constexpr int kRoles = Q8 ? 11 + 4 * kConv : kLook ? 15 : 11;  // warps that are told
  static constexpr uint32_t q_off = 0;
  static constexpr uint32_t k_off = q_off + QT * kTile;
  static constexpr uint32_t v_off = k_off + kKSlots * kTile;
  static constexpr uint32_t stage_off = v_off + kVSlots * kTile;
  static constexpr uint32_t exps_off = stage_off + kStages * kStageBytes;  // [kExps][2][128]
  // [kMeta] int2: the exponent bytes of K and V, and bit 8: there are rows further below than that
  static constexpr uint32_t meta_off = exps_off + (Q8 ? kExps * 256 : 0);
  static constexpr uint32_t stat_off = meta_off + kMeta * 8;               // [2][2][128] float2
  static constexpr uint32_t par_off = stat_off + 2 * 2 * 128 * 8;          // [2][256]
  static constexpr uint32_t bad_off = par_off + 2 * PA_TREE_MAX_TOKENS;    // [kBad][words]
  static constexpr uint32_t bars_off = bad_off + kBad * kTreeWords * 4;
  static constexpr int kBars = kLanded + kStages + 2 * kKSlots + 2 * kVSlots + kMeta + 2 * kExps + 15 + 2 * kAhead +
                               (WIN ? 2 : 0) + (kLook ? kVSlots + 2 : 0);
  using Whole = std::conditional_t<WIN, WindowTile, TreeTile>;
  using Tile = std::conditional_t<SEG, TreeSegment<Whole>, Whole>;
  using Walk = std::conditional_t<WIN, WindowWalk<kTok, 64, kRows, kLead>, TreeWalk<kTok, kRows, kLead>>;
  using Place = TreePlace<Walk, Tile>;
  static constexpr uint32_t tile_off = (bars_off + kBars * 8 + 15) & ~15u;  // [kAhead] row tiles
  static constexpr uint32_t place_off = (tile_off + kAhead * sizeof(Tile) + 15) & ~15u;
  static constexpr uint32_t tmem_off = (place_off + sizeof(Place) + 15) & ~15u;
  static constexpr uint32_t bytes = tmem_off + 16 + 1024;
  static_assert(bytes <= kTcMaxSmem, "shared memory");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
  const uint32_t n = ok ? 16 : 0;  // 0: the 16 bytes are zeroed
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// tree_wait for two barriers at once.
__device__ __forceinline__ bool tree_wait2(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, uint32_t limit) {
  const uint32_t t0 = clock();
#pragma unroll 1
  do {
    if (__all_sync(0xffffffffu, mbar_try_wait(a, pa) & mbar_try_wait(b, pb))) return true;
  } while (__all_sync(0xffffffffu, uint32_t(clock()) - t0 <= limit));
  return false;
}

// A value that is the same in every lane, said so in a way that the compiler
// believes: tcgen05 instructions take their addresses and descriptors from
// uniform registers, and for a value that it must take for divergent it emits a loop
// over the lanes around each of them.
__device__ __forceinline__ uint32_t uni(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ int uni_from(int x, int lane) { return __shfl_sync(0xffffffffu, x, lane); }

// One lane of the warp, in a form that keeps what it issues uniform.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}

// Two fp32 operations in one instruction, and the largest of three.
__device__ __forceinline__ float2 fma_pair(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add_pair(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      " add.rn.f32x2 d, a, b;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Barrier of the eight softmax warps: whether any thread's `pred` holds.
__device__ __forceinline__ bool tree_softmax_bar(bool pred = false) {
  __syncwarp();  // (the barrier wants the warp converged)
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n"
      " bar.red.or.pred q, 1, 256, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(r)
      : "r"(uint32_t(pred))
      : "memory");
  return r != 0;
}

__device__ __forceinline__ uint32_t hmul2u(uint32_t a, uint32_t f) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&f));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Nonzero if one of four e4m3 codes is a NaN.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// An fp16 V tile [HD / 64][128 rows][128 B] before its product (N threads, this one the `lane`-th): rows
// [lo, hi) become 0;
template <int H2, int N = 32>
__device__ __forceinline__ void zero_v_rows(uint8_t* vb, int lo, int hi, int lane) {
  for (int at = lane; at < (hi - lo) * 8 * H2; at += N) {
    const int r = lo + at / (8 * H2), ch = at % (8 * H2);
    *reinterpret_cast<uint4*>(vb + (ch >> 3) * (128 * 128) + r * 128 + (ch & 7) * 16) = make_uint4(0, 0, 0, 0);
  }
}

// non-finite elements of rows [lo, hi) become 0, and `flag` is told their rows.
template <int H2, int N = 32, class Flag>
__device__ __forceinline__ void clear_v_rows(uint8_t* vb, int lo, int hi, int lane, Flag flag) {
  constexpr uint32_t HALF = 128 * 128;
  constexpr int B = 8;  // chunks a lane has in registers at a time
  for (int at0 = lane; at0 < (hi - lo) * 8 * H2; at0 += N * B) {
    uint4 v[B];
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const int at = at0 + N * k, r = lo + at / (8 * H2), ch = at % (8 * H2);
      v[k] = make_uint4(0, 0, 0, 0);
      if (r < hi) v[k] = lds128(vb + (ch >> 3) * HALF + r * 128 + (ch & 7) * 16);
    }
    // zero times anything finite is zero: one product a word tells whether there is something to look for
    __half2 sum = __float2half2_rn(0.f);
    const __half2 zero = sum;
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const __half2* h = reinterpret_cast<const __half2*>(&v[k]);
#pragma unroll
      for (int j = 0; j < 4; ++j) sum = __hfma2(h[j], zero, sum);
    }
    if (__hbeq2(sum, zero)) continue;
#pragma unroll
    for (int k = 0; k < B; ++k) {
      bool hit = clear_nonfinite<false>(v[k].x);
      hit |= clear_nonfinite<false>(v[k].y);
      hit |= clear_nonfinite<false>(v[k].z);
      hit |= clear_nonfinite<false>(v[k].w);
      if (hit) {
        const int at = at0 + N * k, r = lo + at / (8 * H2), ch = at % (8 * H2);
        *reinterpret_cast<uint4*>(vb + (ch >> 3) * HALF + r * 128 + (ch & 7) * 16) = v[k];
        flag(r);
      }
    }
  }
}

// Rows from `hi` become 0, and non-finite elements of rows [lo, hi), drafts row + a0,
// become 0 and are flagged. Rare, hence not inlined.
template <int H2>
__device__ __noinline__ void clean_v_tile(uint8_t* vb, int lo, int hi, int a0, uint32_t* bad, int lane) {
  zero_v_rows<H2>(vb, hi, 128, lane);
  clear_v_rows<H2>(vb, lo, hi, lane, [&](int r) {
    const int a = a0 + r;
    atomicOr(&bad[(a >> 5) % kTreeWords], 1u << (a & 31));
  });
  fence_proxy_async();
  __syncwarp();
}

// (WIN) Of the 64 rows from row0 on, the first one key0's, of which some are not seen by every row of the
// tile: those that no row attends become 0, behind its last token and before the first row's window; of
// those that some attend the non-finite elements do, under a flag (four warps; `lane` of their 128).
// p0: the place of the tile's first token.
template <int H2>
__device__ __forceinline__ void clean_v_window(uint8_t* vb, const WindowTile& t, int p0, int sinks, int row0, int key0,
                                               uint32_t* bad, int lane) {
  const auto row = [&](int key) { return row0 + min(max(key - key0, 0), 64); };
  const auto flag = [&](int) { atomicOr(bad, 1u); };
  // two ranges of each kind, by one loop's code each
#pragma unroll 1
  for (int upper = 0; upper < 2; ++upper) {
    zero_v_rows<H2, 128>(vb, row(upper ? t.L : sinks), upper ? row0 + 64 : row(t.lo), lane);
    clear_v_rows<H2, 128>(vb, row(upper ? p0 + 1 : max(t.lo, sinks)), row(upper ? t.L : min(t.lo1, p0 + 1)), lane,
                          flag);
  }
  fence_proxy_async();
  __syncwarp();
}

// Which of 32 columns a row attends, the first one being draft a0 (negative: prefix) of its sequence:
// of `seen`, its bits, or of a chain, whose row is draft `qi`.
__device__ __forceinline__ uint32_t tree_attends(const uint32_t* seen, int qi, int a0) {
  if (a0 <= -32) return ~0u;
  if (!seen) {
    const int n = qi - a0 + 1;  // columns up to the row's own
    return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1;
  }
  // bits a0 .. a0 + 31 of (ones below 0, then the row's drafts)
  const int q = a0 >> 5;
  const uint32_t lo = q < 0 ? ~0u : q < kTreeWords ? seen[q] : 0u;
  const uint32_t hi = q + 1 < kTreeWords ? seen[q + 1] : 0u;
  return __funnelshift_r(lo, hi, a0 & 31);
}

// The scores of a job some of whose keys lie further below the tile's exponents than they were
// brought up to, 64 columns of S in TMEM, become base-2 exponents of weights in place: s_j + v_j, with
// s_j = S_j * scale * 2^k_j and k_j, v_j what is left of the exponents in `exps` (V's 128 bytes behind
// K's). `left` columns lie in the context, the first is draft a0. *own: the largest s_j that
// the row attends and the sum of 2^(s_j - it). Rare, hence not inlined and a loop of 16 columns.
// (WIN: the row's token stands at qi, the first column is the key a0.)
template <int SPREAD_K, int SPREAD_V, bool WIN>
__device__ __noinline__ void tree_apart(const TreeParams& P, uint32_t sbuf, const uint8_t* exps, int2 tile, int left,
                                        const uint32_t* seen, int qi, int a0, float2* own) {
  float top = -INFINITY, sum = 0.f;
#pragma unroll 1
  for (int c = 0; c < 64; c += 16) {
    float s[16], most = top;
    uint32_t x[16];
    __syncwarp();
    tmem_ld<16>(sbuf + c, s);
    tmem_wait_ld();
    const int col = a0 + (c & 32);
    const uint32_t bits = (WIN ? window_bits(P, qi, col) : tree_attends(seen, qi, col)) >> (c & 16);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      int k = (tile.x & 255) - kExpBias, v = (tile.y & 255) - kExpBias;
      if (c + j < left) {  // (exponents behind the context: anything)
        k = min(k, max(int(exps[c + j]), kExpLeastByte) - kExpBias + SPREAD_K);
        v = min(v, max(int(exps[c + j + 128]), kExpLeastByte) - kExpBias + SPREAD_V);
      }
      s[j] *= fmaxf(P.scale_log2 * pow2(k), FLT_MIN);
      x[j] = __float_as_uint(s[j] + float(v));
      if (!(bits >> j & 1)) s[j] = -INFINITY;
      most = fmaxf(most, s[j]);
    }
    const float ref = most == -INFINITY ? 0.f : most;
    float add = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) add += ex2(s[j] - ref);
    sum = fmaf(sum, ex2(top - ref), add);
    top = most;
    __syncwarp();
    tmem_st16u(sbuf + c, x);
  }
  __syncwarp();
  tmem_wait_st();
  *own = make_float2(top, sum);
}

template <int HD, bool Q8, int QT, bool WIN, bool SEG>
__global__ void __launch_bounds__(TreeTc<HD, Q8, QT, WIN, SEG>::kThreads, 1)
    tree_tc_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                   const __grid_constant__ std::conditional_t<WIN, CUtensorMap, int> tmq,
                   const __grid_constant__ TreeParams P, const __grid_constant__ TreeSplit S) {
  using Cfg = TreeTc<HD, Q8, QT, WIN, SEG>;
  using Tile = typename Cfg::Tile;
  constexpr int TOK = Cfg::kTok, H2 = Cfg::kHalves, KS = Cfg::kKSlots, VS = Cfg::kVSlots;
  constexpr uint32_t kTmemCols = 512;
  constexpr uint32_t kIdescQK = mma_idesc(128, TOK, 0, 0);
  constexpr uint32_t kIdescPV = mma_idesc(128, HD, 0, 1);
  constexpr unsigned FULL = 0xffffffffu;
  extern __shared__ uint8_t smem_raw[];
  // (offset, not masked: the compiler keeps seeing shared memory behind the pointer)
  uint8_t* smem = smem_raw + (-smem_u32(smem_raw) & 1023u);
  const int tid = threadIdx.x, lane = tid & 31, warp = int(uni(tid >> 5));
  uint8_t* q_s = smem + Cfg::q_off;
  uint8_t* kring = smem + Cfg::k_off;
  uint8_t* vring = smem + Cfg::v_off;
  int2* meta = reinterpret_cast<int2*>(smem + Cfg::meta_off);
  uint32_t* bad_s = reinterpret_cast<uint32_t*>(smem + Cfg::bad_off);
  uint64_t* sfull = reinterpret_cast<uint64_t*>(smem + Cfg::bars_off);  // [K, V][round][part]
  uint64_t* sempty = sfull + Cfg::kLanded;  // [stage]
  uint64_t* kfull = sempty + Cfg::kStages;
  uint64_t* kempty = kfull + KS;
  uint64_t* vfull = kempty + KS;
  uint64_t* vempty = vfull + VS;
  uint64_t* meta_full = vempty + VS;
  uint64_t* exps_full = meta_full + Cfg::kMeta;      // [K, V][kExps]
  uint64_t* tile_full = exps_full + 2 * Cfg::kExps;  // a row tile told to the roles
  uint64_t* tile_empty = tile_full + Cfg::kAhead;
  // (of a job: [g][y], y the key tile's parity for QT = 1, its half for QT = 2)
  uint64_t* s_full = tile_empty + Cfg::kAhead;  // [x] S written
  uint64_t* p_full = s_full + 2;              // [g][y] P written, O_g rescaled
  uint64_t* pv_done = s_full + 6;             // [g][y] O_g += P V complete
  uint64_t* o_full = s_full + 10;             // [g] the row tile's last PV_g complete
  uint64_t* q_empty = s_full + 12;            // the row tile's last S complete
  uint64_t* o_free = s_full + 13;             // both O read by the softmax warps
  uint64_t* all_done = s_full + 14;
  uint64_t* q_full = s_full + 15;             // (WIN) the queries, by TMA
  uint64_t* o_free1 = s_full + 16;            // (WIN, QT = 2) O_1 read, o_free O_0 alone
  uint64_t* stat_full = s_full + 17;          // (kLook) [row tile's parity] maxima and sums told
  uint64_t* vready = s_full + 19;             // (kLook) [slot] V looked through
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cfg::tmem_off);
  const int worker = blockIdx.x;

  if (tid == 0) {
    prefetch_tensormap(&tmk);
    prefetch_tensormap(&tmv);
    for (int i = 0; i < Cfg::kLanded; ++i) mbar_init(&sfull[i], 1);
    for (int i = 0; i < Cfg::kStages; ++i) mbar_init(&sempty[i], Cfg::kConv);
    for (int i = 0; i < KS; ++i) {
      mbar_init(&kfull[i], Q8 ? 2 * Cfg::kConv : 1);
      mbar_init(&kempty[i], 1);
    }
    for (int i = 0; i < VS; ++i) {
      mbar_init(&vfull[i], Q8 ? 2 * Cfg::kConv : 1);
      mbar_init(&vempty[i], 1);
      if (Cfg::kLook) mbar_init(&vready[i], 4);
    }
    for (int i = 0; i < Cfg::kMeta; ++i) mbar_init(&meta_full[i], 2);
    for (int i = 0; i < 2 * Cfg::kExps; ++i) mbar_init(&exps_full[i], 1);
    for (int i = 0; i < Cfg::kAhead; ++i) {
      mbar_init(&tile_full[i], 1);
      mbar_init(&tile_empty[i], Cfg::kRoles);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(&s_full[g], 1);
      mbar_init(&o_full[g], 1);
    }
    mbar_init(q_empty, 1);
    mbar_init(o_free, (WIN && QT == 2 ? 4 : 8) + (Cfg::kShare ? 4 : 0));
    if (WIN) mbar_init(o_free1, 4 + (Cfg::kShare ? 4 : 0));
    mbar_init(all_done, WIN ? 1 : 2);
    if (WIN) mbar_init(q_full, 1);
    if (Cfg::kLook) {
      mbar_init(&stat_full[0], 8);
      mbar_init(&stat_full[1], 8);
    }
    fence_barrier_init();
  }
  if (tid < Cfg::kBad * kTreeWords) bad_s[tid] = 0;
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(tmem_slot)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uni(*tmem_slot);
  const uint32_t tmem_s = tmem, tmem_o = tmem + 256;
  const int G = P.group, bs = P.block_size;

  // The row tiles, as warp 3 finds them on the line, told to the other roles through
  // a ring (one reading of the lengths for the whole CTA); q < 0 ends them.
  Tile* told = reinterpret_cast<Tile*>(smem + Cfg::tile_off);
  int heard = 0;  // row tiles begun
  auto next_tile = [&](Tile& t) {
    __syncwarp();
    if (heard > 0 && lane == 0) mbar_arrive(&tile_empty[(heard - 1) % Cfg::kAhead]);
    const int at = heard % Cfg::kAhead;
    if (!tree_wait(&tile_full[at], (heard / Cfg::kAhead) & 1, P.wait_limit)) return false;
    t = told[at];
    ++heard;
    return t.q >= 0;
  };
  // Key tiles of a row tile: the keys past its last row's own position are no
  // row's, so a tile of early rows (or a worker's share of one) may have fewer
  // units than the line counts, or none.
  auto key_tiles = [&](const Tile& w) {
    if constexpr (WIN) return w.s1 - w.s0;  // (counted as they are)
    const int last = min(w.q - 1, (w.r0 + Cfg::kRows - 1) / G);
    const int units = (w.L - w.q + last + TOK) / TOK;
    return max(0, min(w.s1, units) - w.s0);
  };
  // The first key of a half of a row tile's unit, and whether some of n keys are not seen by all of its rows.
  auto key_of = [&](const Tile& w, int u, int half) {
    if constexpr (WIN) return w.chunk(2 * u + half) * 64;
    else return u * TOK + half * 64;
  };
  // (first: the place of its first token, WIN; of the first token of all)
  auto edge_at = [&](const Tile& w, int first, int key, int n) {
    if constexpr (WIN) return key + n > first + 1 || (key < w.lo1 && key + n > P.sinks);
    else return key + n > first;
  };
  // The token of a row of a row tile, and its head of the group.
  auto token_of = [&](const Tile& w, int row) {
    if constexpr (WIN) return w.token(P, row);
    else return (w.r0 + row) / G;
  };
  auto head_of = [&](const Tile& w, int row, int token) { return w.r0 + row - token * G; };
  // Where the rows of four lanes next to one another go to in the output, this lane's to `mine`; null for
  // rows that are not.
  auto rows_out = [&](__half* mine, __half* (&dst)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint64_t a = __shfl_sync(FULL, reinterpret_cast<uint64_t>(mine), (lane & ~3) + k);
      dst[k] = a ? reinterpret_cast<__half*>(a) + (lane & 3) * 8 : nullptr;
    }
  };
  // 32 columns of a row a thread in fp16. Four lanes next to one another hold four rows, 64 bytes each, and
  // exchange them by quarters, so that a store writes eight rows' 64 bytes rather than 16 of 32
  // rows (which took 3.2 us of a tile of 256 rows, 2 so).
  auto store32 = [&](uint32_t (&h)[4][4], __half* const (&dst)[4], int col) {  // [eight columns][pairs of them]
#pragma unroll
    for (int bit = 1; bit < 4; bit <<= 1) {
      const bool upper = lane & bit;
#pragma unroll
      for (int a = 0; a < 4; ++a) {
        if (a & bit) continue;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t give = upper ? h[a][k] : h[a | bit][k];
          const uint32_t got = __shfl_xor_sync(FULL, give, bit);
          if (upper) h[a][k] = got; else h[a | bit][k] = got;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (dst[k]) *reinterpret_cast<uint4*>(dst[k] + col) = make_uint4(h[k][0], h[k][1], h[k][2], h[k][3]);
  };
  auto pack32 = [&](const float* o, float inv, uint32_t (&h)[4][4]) {
#pragma unroll
    for (int k = 0; k < 16; ++k) h[k / 4][k % 4] = pack_half2(o[2 * k] * inv, o[2 * k + 1] * inv);
  };
  // The phase of key tile n's S and jobs on their barriers.
  auto phase_of = [](int n) { return QT == 2 ? n & 1 : n >> 1 & 1; };
  bool ok = true;

  if (warp == 0 || warp == 2) {
    // ================= copies: keys (warp 0), values (warp 2) =================
    // Lane l has piece l of every key tile, box keys that lie in one block: its place
    // in the block table moves on by additions, and the next tile's entry is read
    // before this one's slots are waited for.
    const int box = min(bs & -bs, 64), pieces = TOK / box, step_b = TOK / bs, step_o = TOK % bs;
    // (WIN: the next row tiles read the window again)
    const uint64_t pol = WIN && QT == 2 ? policy_evict_last() : policy_evict_first();
    const bool is_k = warp == 0;
    const CUtensorMap* map = is_k ? &tmk : &tmv;
    const uint8_t* exps_of = is_k ? P.key_exps : P.value_exps;
    // the ring: stages of 64 keys (8-bit cache) or tiles
    const int nslots = Q8 ? (is_k ? Cfg::kKStages : Cfg::kVStages) : is_k ? KS : VS;
    uint64_t* fulls = Q8 ? sfull + (is_k ? 0 : 2 * Cfg::kKRounds) : is_k ? kfull : vfull;
    const int rounds = is_k ? Cfg::kKRounds : Cfg::kVRounds;
    uint64_t* empties = Q8 ? sempty + (is_k ? 0 : Cfg::kKStages) : is_k ? kempty : vempty;
    uint8_t* ring = Q8 ? smem + Cfg::stage_off + (is_k ? 0 : Cfg::kKStages) * Cfg::kStageBytes : is_k ? kring : vring;
    const int half = pieces / 2, part = lane >= half ? 1 : 0;
    int n = 0, filled = 0;     // key tiles, and stages or tiles filled, so far
    int slot = 0, phase = 0;   // of the next stage or tile
    int round = 0;             // of the next key tile's barriers
    Tile t;
    while (ok && next_tile(t)) {
      const int tiles = key_tiles(t);
      const int32_t* table = P.block_tables + int64_t(t.b) * P.max_blocks_per_seq;
      const auto wanted = [&](int key) {
        bool w = lane < pieces && key < t.L;
        if constexpr (WIN) w = w && !window_hidden(P, t.lo, key, box);
        return w;
      };
      int key = key_of(t, t.s0, part) + (lane - part * half) * box, blk = key / bs, off = key - blk * bs;
      int id = tiles > 0 && wanted(key) ? table[blk] : -1;
      for (int i = 0; i < tiles; ++i, ++n) {
        const bool want = wanted(key), there = want && id >= 0 && id < P.num_blocks;
        if (want && !there) set_status(P.status, PA_STATUS_BIT_BLOCK_INDEX);
        const unsigned valid = __ballot_sync(FULL, there);
        const int row = id * bs + off, id_now = id, off_now = off;
        key += TOK;
        blk += step_b;
        off += step_o;
        if (off >= bs) {
          off -= bs;
          ++blk;
        }
        if constexpr (WIN) {
          const int c = 2 * (t.s0 + i) + part;
          if (t.skip && c < t.far && c + 2 >= t.far) {  // from the sinks to the window
            key += t.skip * 64;
            blk = key / bs;
            off = key - blk * bs;
          }
        }
        id = i + 1 < tiles && wanted(key) ? table[blk] : -1;
        if constexpr (Q8) {
          const int slot1 = slot + 1 == nslots ? 0 : slot + 1, phase1 = slot1 == 0 ? phase ^ 1 : phase;
          const int em = n % Cfg::kExps;
          uint64_t* efull = &exps_full[(is_k ? 0 : Cfg::kExps) + em];
          const int64_t eat = (int64_t(id_now) * P.kv_heads + t.kvh) * bs + off_now;
          uint8_t* dst = ring + (part ? slot1 : slot) * Cfg::kStageBytes + (lane - part * half) * box * HD;
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            uint64_t* full = &fulls[2 * round + p];
            if (!tree_wait(&empties[p ? slot1 : slot], (p ? phase1 : phase) ^ 1, P.wait_limit)) {
              ok = false;
              break;
            }
            if (lane == 0) {
              const uint32_t bytes = __popc(valid >> (p * half) & ((1u << half) - 1)) * box * HD;
              if (bytes) mbar_arrive_expect_tx(full, bytes); else mbar_arrive(full);
            }
            // (the exponents' slot was last read kExps tiles ago, long before what was waited for)
            if (p == 0 && lane == 1) {
              const uint32_t bytes = __popc(valid) * box;
              if (bytes) mbar_arrive_expect_tx(efull, bytes); else mbar_arrive(efull);
            }
            __syncwarp();
            if (there && part == p) tma_load_2d(dst, map, full, t.kvh * HD, row, pol);
            if (p == 0 && there)
              bulk_load(smem + Cfg::exps_off + em * 256 + (is_k ? 0 : 128) + lane * box, exps_of + eat, box, efull);
            __syncwarp();
            ++filled;
          }
          if (!ok) break;
          if (++round == rounds) round = 0;
          slot = slot1 + 1 == nslots ? 0 : slot1 + 1;
          phase = slot == 0 ? phase1 ^ 1 : phase1;
        } else {
          if (!tree_wait(&empties[slot], phase ^ 1, P.wait_limit)) {
            ok = false;
            break;
          }
          uint64_t* full = &fulls[slot];
          if (lane == 0) {
            const uint32_t bytes = __popc(valid) * box * 128 * H2;
            if (bytes) mbar_arrive_expect_tx(full, bytes); else mbar_arrive(full);
          }
          __syncwarp();
          if (there)
            for (int h = 0; h < H2; ++h)
              tma_load_3d(ring + slot * Cfg::kTile + h * Cfg::kHalf + lane * box * 128, map, full, 0, row,
                          t.kvh * H2 + h, pol);
          __syncwarp();
          ++filled;
          if (++slot == nslots) {
            slot = 0;
            phase ^= 1;
          }
        }
      }
    }
    // copies still in flight land before the CTA's memory is given back
    const int nfulls = Q8 ? 2 * rounds : nslots;
    for (int i = 0; i < nfulls; ++i) {
      const int times = filled / nfulls + (i < filled % nfulls ? 1 : 0);
      if (times) tree_wait(&fulls[i], (times - 1) & 1);
    }
    if constexpr (Q8) {
      // (a tile's exponents come with its first part, which the second may not have followed)
      const int with_exps = (filled + 1) / 2;
      for (int i = max(0, with_exps - Cfg::kExps); i < with_exps; ++i)
        tree_wait(&exps_full[(is_k ? 0 : Cfg::kExps) + i % Cfg::kExps], (i / Cfg::kExps) & 1);
    }
  } else if (warp == 1) {
    if constexpr (WIN) {
    // ================= S = Q K^T and O_g += P_g V =================
    // Both products in one order, each S right behind the product that read the P in its columns: the
    // products of one thread are done in their order, so no wait stands between them. (256 rows x 128 keys
    // in 1.70 us; 1.85 with S issued by warp 3, behind a wait.) The whole warp waits and counts, one
    // lane issues.
    const uint64_t dq = smem_desc(smem_u32(q_s), 16, 1024), dk = smem_desc(smem_u32(kring), 16, 1024);
    const uint64_t dv = smem_desc(smem_u32(vring), Cfg::kHalf, 1024);
    uint64_t* vcome = Cfg::kLook ? vready : vfull;
    int tile = 0, n0 = 0;  // row tiles and key tiles so far
    int kslot = 0, kphase = 0, vslot = 0, vphase = 0;
    Tile t;
    while (ok && next_tile(t)) {
      const int tiles = uni(key_tiles(t));
      // S of key tile i, of query tile g (QT = 2)
      auto scores = [&](int i, int g) {
        if (g == 0 && !tree_wait(&kfull[kslot], kphase, P.wait_limit)) {
          ok = false;
          return;
        }
        const int x = QT == 2 ? g : (n0 + i) & 1;
        const bool last = i + 1 == tiles && g == QT - 1;
        const uint64_t bk = dk + uint32_t(kslot * (Cfg::kTile >> 4));
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int h = 0; h < H2; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc_mma(tmem_s + x * 128, dq + g * (Cfg::kTile >> 4) + ((h * Cfg::kHalf + k * 32) >> 4),
                     bk + ((h * Cfg::kHalf + k * 32) >> 4), kIdescQK, (h | k) != 0);
          tc_commit(&s_full[x]);
          if (g == QT - 1) tc_commit(&kempty[kslot]);
          if (last) tc_commit(q_empty);  // the queries may be replaced
        }
        __syncwarp();
        if (g == QT - 1 && ++kslot == KS) {
          kslot = 0;
          kphase ^= 1;
        }
      };
      if (!tree_wait(q_full, tile & 1, P.wait_limit)) {
        ok = false;
        break;
      }
      scores(0, 0);
      if (ok && QT == 2) scores(0, 1);
      if (ok && QT == 1 && tiles > 1) scores(1, 0);
      for (int i = 0; i < tiles && ok; ++i) {
        const int n = n0 + i, phase = phase_of(n);
        const bool last = i + 1 == tiles;
        if (!tree_wait(&vcome[vslot], vphase, P.wait_limit)) { ok = false; break; }
#pragma unroll
        for (int j = 0; j < 2 * QT; ++j) {
          const int g = j & 1, hf = QT == 2 ? j >> 1 : g, y = QT == 2 ? hf : n & 1;
          // the last row tile's O has been read before the first product overwrites it
          if (i == 0 && tile > 0 && (QT == 2 ? hf == 0 : g == 0) &&
              !tree_wait(QT == 2 && g ? o_free1 : o_free, (tile - 1) & 1, P.wait_limit)) {
            ok = false;
            break;
          }
          if (!tree_wait(&p_full[2 * g + y], phase, P.wait_limit)) { ok = false; break; }
          const uint64_t bv = dv + uint32_t(vslot * (Cfg::kTile >> 4) + hf * (8192 >> 4));
          const uint32_t p_col = tmem_s + (QT == 2 ? g : n & 1) * 128 + hf * 64;
          const bool more = i != 0 || (QT == 2 && hf);
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              tc_mma_tmem_a(tmem_o + g * 128, p_col + k * 8, bv + (k * 2048 >> 4), kIdescPV, k || more);
            tc_commit(&pv_done[2 * g + y]);
            if (j == 2 * QT - 1) tc_commit(&vempty[vslot]);
            if (last && (QT == 1 || hf)) tc_commit(&o_full[g]);
          }
          __syncwarp();
          if (QT == 2 && hf == 1 && !last) scores(i + 1, g);
          if (!ok) break;
        }
        if (QT == 1 && ok && i + 2 < tiles) scores(i + 2, 0);
        if (++vslot == VS) {
          vslot = 0;
          vphase ^= 1;
        }
      }
      n0 += tiles;
      ++tile;
    }
    if (elect_one()) tc_commit(all_done);
    __syncwarp();
    } else {
    // ================= O_g += P_g V =================
    // Per key tile the two chains' products in turn (QT = 2: of its halves in turn).
    // The whole warp waits and counts, one lane issues: what the instructions take
    // from uniform registers then stays in them. Descriptors are a base and an offset in
    // 16-byte units (the address field, in the low bits, does not overflow).
    const uint64_t dv = smem_desc(smem_u32(vring), Cfg::kHalf, 1024);
    int tile = 0, n0 = 0, vslot = 0, vphase = 0;  // row tiles and key tiles so far; the next V tile
    Tile t;
    while (ok && next_tile(t)) {
      const int tiles = uni(key_tiles(t));
      const int q_len = uni(t.q), prefix = uni(t.L) - q_len, s0 = uni(t.s0);
      auto pv = [&](int g, int y, int hf, uint32_t p_col, bool more, bool tile_done, bool last) {
        const uint64_t bv = dv + uint32_t(vslot * (Cfg::kTile >> 4) + hf * (8192 >> 4));
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            tc_mma_tmem_a(tmem_o + g * 128, p_col + k * 8, bv + (k * 2048 >> 4), kIdescPV, k || more);
          tc_commit(&pv_done[2 * g + y]);
          if (tile_done) tc_commit(&vempty[vslot]);
          if (last) tc_commit(&o_full[g]);
        }
        __syncwarp();
      };
      // the last row tile's O has been read before the first product overwrites it
      if (tile > 0 && !tree_wait(o_free, (tile - 1) & 1, P.wait_limit)) ok = false;
      for (int i = 0; i < tiles && ok; ++i) {
        const int n = n0 + i, phase = phase_of(n);
        const bool last = i + 1 == tiles;
        if (!tree_wait(&vfull[vslot], vphase, P.wait_limit)) { ok = false; break; }
        if constexpr (!Q8) {
          // Rows behind the context may hold anything and become 0; non-finite
          // elements of the drafts' rows leave the product
          const int key0 = (s0 + i) * TOK;
          if (key0 + TOK > prefix)
            clean_v_tile<H2>(vring + vslot * Cfg::kTile, max(prefix - key0, 0), min(prefix + q_len - key0, TOK),
                             key0 - prefix, bad_s + (tile % Cfg::kBad) * kTreeWords, lane);
        }
#pragma unroll
        for (int j = 0; j < 2 * QT; ++j) {
          const int g = j & 1, hf = QT == 2 ? j >> 1 : g, y = QT == 2 ? hf : n & 1;
          if (!tree_wait(&p_full[2 * g + y], phase, P.wait_limit)) { ok = false; break; }
          pv(g, y, hf, tmem_s + (QT == 2 ? g : n & 1) * 128 + hf * 64, i != 0 || (QT == 2 && hf), j == 2 * QT - 1,
             last && (QT == 1 || hf));
        }
        if (++vslot == VS) {
          vslot = 0;
          vphase ^= 1;
        }
      }
      n0 += tiles;
      ++tile;
    }
    if (elect_one()) tc_commit(all_done);
    __syncwarp();
    }
  } else if (warp == 3) {
    if constexpr (WIN) {
    // ================= row tiles and their queries =================
    int told_n = 0, tile = 0;  // row tiles told, begun
    bool by_tma = false;
    if (lane == 0) S.join[worker].parts = 0;  // no divided tile yet
    typename Cfg::Place* place = reinterpret_cast<typename Cfg::Place*>(smem + Cfg::place_off);
    Tile t, following;
    tree_begin(P, S, place, worker, lane);
    auto tell = [&]() {  // finds the next row tile and tells it; q < 0: there is none
      const bool some = tree_next(P, S, place);
      following = place->tile;
      if (!some) following.q = -1;
      const int at = told_n % Cfg::kAhead;
      if (!tree_wait(&tile_empty[at], ((told_n / Cfg::kAhead) & 1) ^ 1, P.wait_limit)) {
        ok = false;
        return;
      }
      if (lane == 0) {
        told[at] = following;
        if (following.q >= 0 && following.parts) tree_note(S, worker, following);
        mbar_arrive(&tile_full[at]);
      }
      __syncwarp();
      ++told_n;
      if (place->walk.u >= place->walk.u1) launch_dependents();  // the worker's last tile is known
    };
    tell();
    while (ok && following.q >= 0) {
      t = following;
      // the queries, once the last row tile's S are complete
      if (tile > 0 && !tree_wait(q_empty, (tile - 1) & 1, P.wait_limit)) {
        ok = false;
        break;
      }
      // Whole tokens whose heads make up 128 rows: one box of 64 dims of each half tile. Tokens behind
      // the tile's last come along (their rows are not looked at), zeros behind the last of all.
      by_tma = 128 % G == 0;
      if (by_tma) {
        if (lane == 0) {
          const uint64_t keep = policy_evict_first();
          mbar_arrive_expect_tx(q_full, QT * Cfg::kTile);
#pragma unroll
          for (int x = 0; x < QT; ++x)
#pragma unroll
            for (int h = 0; h < H2; ++h)
              tma_load_3d(q_s + x * Cfg::kTile + h * Cfg::kHalf, &tmq, q_full, h * 64, t.kvh * G,
                          t.q_start + t.r0 / G + x * (128 / G), keep);
        }
        __syncwarp();
      } else {
        constexpr int CH = HD / 8, RPI = 32 / CH;  // 16-byte chunks of a row, rows of a copy
        const int ch = lane % CH;
        const uint32_t base = smem_u32(q_s) + (ch >> 3) * Cfg::kHalf;
#pragma unroll 1
        for (int r0 = 0; r0 < Cfg::kRows; r0 += 32) {
          // lane l finds row r0 + l of the query tensor
          const int r = t.r0 + r0 + lane, i = r / G;
          const int64_t tok = int64_t(t.q_start) + i;
          const int from = i < t.q && tok < P.tokens ? int(tok * P.num_heads + t.kvh * G + r % G) : -1;
#pragma unroll
          for (int k = 0; k < 32 / RPI; ++k) {
            const int row = r0 + k * RPI + lane / CH;
            const int src = __shfl_sync(FULL, from, k * RPI + lane / CH);
            cp_async16(base + (row >> 7) * Cfg::kTile + (row & 127) * 128 + (((ch & 7) ^ (row & 7)) << 4),
                       P.query + int64_t(max(src, 0)) * HD + ch * 8, src >= 0);
          }
        }
        cp_async_commit();
        cp_async_wait<0>();
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
        __syncwarp();
      }
      tell();  // the next row tile, while these queries come
      ++tile;
    }
    // (landed before the CTA's memory is given back)
    if (by_tma) tree_wait(q_full, (tile - 1) & 1);
    } else {
    // ================= row tiles, their queries, S = Q K^T =================
    const uint64_t dq = smem_desc(smem_u32(q_s), 16, 1024), dk = smem_desc(smem_u32(kring), 16, 1024);
    int told_n = 0, tile = 0, n = 0, kslot = 0, kphase = 0;  // tiles told, begun; key tiles; the next K tile
    if (lane == 0) S.join[worker].parts = 0;                 // no divided tile yet
    typename Cfg::Place* place = reinterpret_cast<typename Cfg::Place*>(smem + Cfg::place_off);
    Tile t, following;
    tree_begin(P, S, place, worker, lane);
    auto tell = [&]() {  // finds the next row tile and tells it; q < 0: there is none
      const bool some = tree_next(P, S, place);
      following = place->tile;
      if (!some) following.q = -1;
      const int at = told_n % Cfg::kAhead;
      if (!tree_wait(&tile_empty[at], ((told_n / Cfg::kAhead) & 1) ^ 1, P.wait_limit)) {
        ok = false;
        return;
      }
      if (lane == 0) {
        told[at] = following;
        if (following.q >= 0 && following.parts) tree_note(S, worker, following);
        mbar_arrive(&tile_full[at]);
      }
      __syncwarp();
      ++told_n;
      if (place->walk.u >= place->walk.u1) launch_dependents();  // the worker's last tile is known
    };
    tell();
    while (ok && following.q >= 0) {
      t = following;
      const int tiles = uni(key_tiles(t));
      // the queries, once the last row tile's S are complete
      if (tile > 0 && !tree_wait(q_empty, (tile - 1) & 1, P.wait_limit)) {
        ok = false;
        break;
      }
      constexpr int CH = HD / 8, RPI = 32 / CH;  // 16-byte chunks of a row, rows of a copy
      const int ch = lane % CH;
      const uint32_t base = smem_u32(q_s) + (ch >> 3) * Cfg::kHalf;
#pragma unroll 1
      for (int r0 = 0; r0 < Cfg::kRows; r0 += 32) {
        // lane l finds row r0 + l of the query tensor
        const int r = t.r0 + r0 + lane, i = r / G;
        const int64_t tok = int64_t(t.q_start) + i;
        const int from = i < t.q && tok < P.tokens ? int(tok * P.num_heads + t.kvh * G + r % G) : -1;
#pragma unroll
        for (int k = 0; k < 32 / RPI; ++k) {
          const int row = r0 + k * RPI + lane / CH;
          const int src = __shfl_sync(FULL, from, k * RPI + lane / CH);
          cp_async16(base + (row >> 7) * Cfg::kTile + (row & 127) * 128 + (((ch & 7) ^ (row & 7)) << 4),
                     P.query + int64_t(max(src, 0)) * HD + ch * 8, src >= 0);
        }
      }
      cp_async_commit();
      tell();  // the next row tile, while the queries come
      cp_async_wait<0>();
      fence_proxy_async();
      __syncwarp();
      for (int i = 0; i < tiles && ok; ++i, ++n) {
        if (!tree_wait(&kfull[kslot], kphase, P.wait_limit)) { ok = false; break; }
        const bool last = i + 1 == tiles;
        const uint64_t bk = dk + uint32_t(kslot * (Cfg::kTile >> 4));
#pragma unroll
        for (int g = 0; g < QT; ++g) {
          // what stood in these columns, the P of two tiles ago (QT = 2: of the last),
          // has been read
          const int x = QT == 2 ? g : n & 1, nb = QT == 2 ? n - 1 : n - 2;
          if (nb >= 0 && !tree_wait2(&pv_done[QT == 2 ? 2 * g : x], phase_of(nb), &pv_done[QT == 2 ? 2 * g + 1 : 2 + x],
                                     phase_of(nb), P.wait_limit)) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int h = 0; h < H2; ++h)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                tc_mma(tmem_s + x * 128, dq + g * (Cfg::kTile >> 4) + ((h * Cfg::kHalf + k * 32) >> 4),
                       bk + ((h * Cfg::kHalf + k * 32) >> 4), kIdescQK, (h | k) != 0);
            tc_commit(&s_full[x]);
            if (g == QT - 1) tc_commit(&kempty[kslot]);
            if (g == QT - 1 && last) tc_commit(q_empty);  // the queries may be replaced
          }
          __syncwarp();
        }
        if (++kslot == KS) {
          kslot = 0;
          kphase ^= 1;
        }
      }
      if (tiles == 0) {
        if (elect_one()) tc_commit(q_empty);
        __syncwarp();
      }
      ++tile;
    }
    if (elect_one()) tc_commit(all_done);
    __syncwarp();
    }
  } else if (warp >= 4 && warp < 12) {
    // ================= softmax: group g (warps 4-7, 8-11) is chain g =================
    const int g = (warp - 4) >> 2, quarter = warp & 3, m_lane = quarter * 32 + lane;
    const int tr = (QT == 2 ? g * 128 : 0) + m_lane;  // row of the row tile
    const uint32_t lane_base = uint32_t(quarter * 32) << 16;
    float2* stat = reinterpret_cast<float2*>(smem + Cfg::stat_off);
    int tile = 0, n0 = 0, oc = 0;  // row tiles, key tiles, row tiles with keys
    // Agreed on by both groups, which meet at barriers: that every warp has seen the next row tile told
    // too (next_tile does not wait here), as one whose wait ran out would leave the others at one.
    if (!tree_wait(&tile_full[0], 0, P.wait_limit)) ok = false;
    bool alive = !tree_softmax_bar(!ok);
    Tile t;
    while (alive && next_tile(t)) {
      const int tiles = key_tiles(t), nj = QT * tiles;
      const int prefix = t.L - t.q, qi = token_of(t, tr), head = head_of(t, tr, qi);
      const int64_t tok = int64_t(t.q_start) + qi;
      const bool row_ok = qi < t.q && tok < P.tokens;
      const bool any_row = __any_sync(FULL, row_ok);
      const bool drafts = WIN || (t.s0 + tiles) * TOK > prefix;
      uint32_t bits[WIN ? 1 : kTreeWords] = {};  // the drafts that this row sees (indexed: in local memory)
      if constexpr (!WIN) if (drafts && P.parents) {
        uint8_t* par = smem + Cfg::par_off + (tile & 1) * PA_TREE_MAX_TOKENS;
        for (int i = tid - 128; i < t.q; i += 256) {
          const int up = int64_t(t.q_start) + i < P.tokens ? P.parents[t.q_start + i] : -1;
          const bool fine = up >= -1 && up < i;
          if (!fine) set_status(P.status, PA_STATUS_BIT_TREE);
          par[i] = fine && up >= 0 ? uint8_t(up) : 255;
        }
        tree_softmax_bar();
        if (row_ok) {
          for (int i = qi;; i = par[i]) {
            bits[i >> 5] |= 1u << (i & 31);
            if (par[i] == 255) break;
          }
        }
      }
      // (WIN) the places of the warp's first and last row
      const int rw = (QT == 2 ? g * 128 : 0) + quarter * 32;
      const int pw0 = WIN ? prefix + token_of(t, rw) : 0, pw1 = WIN ? prefix + min(token_of(t, rw + 31), t.q - 1) : 0;
      float m_ref = -INFINITY, l = 0.f;
      for (int m = 0; m < nj && ok; ++m) {
        const int i = QT == 2 ? m >> 1 : m, hf = QT == 2 ? m & 1 : g, n = n0 + i;
        const int y = QT == 2 ? hf : n & 1, x_of_s = QT == 2 ? g : n & 1, phase = phase_of(n);
        const int key0 = key_of(t, t.s0 + i, hf);
        float F = P.scale_log2, ev = 0.f, unscale = 1.f;
        int2 e = make_int2(0, 0);
        if constexpr (Q8) {
          const int k = n % Cfg::kMeta;
          if (!tree_wait(&meta_full[k], (n / Cfg::kMeta) & 1, P.wait_limit)) { ok = false; break; }
          e = meta[k];
          F = fmaxf(F * pow2((e.x & 255) - kExpBias), FLT_MIN);  // (0 times the -inf of a masked score is NaN)
          ev = float((e.y & 255) - kExpBias);
          unscale = pow2(kExpBias - (e.y & 255));
        }
        if (!tree_wait(&s_full[x_of_s], phase, P.wait_limit)) { ok = false; break; }
        tc_fence_after();
        if (WIN && any_row && (key0 > pw1 || (pw0 - key0 - 63 >= P.window && key0 >= P.sinks))) {
          // keys that none of the warp's rows sees: weights of 0
          const uint32_t none[16] = {};
          const uint32_t sbuf = uni(tmem_s + x_of_s * 128 + hf * 64 + lane_base);
          __syncwarp();
          tmem_st16u(sbuf, none);
          tmem_st16u(sbuf + 16, none);
          tmem_wait_st();
        } else if (any_row) {
          __syncwarp();
          const uint32_t sbuf = uni(tmem_s + x_of_s * 128 + hf * 64 + lane_base);
          float2 own;  // of keys with exponents of their own: the largest score, the sum
          if (Q8 && ((e.x | e.y) & 256)) {
            const int em = n % Cfg::kExps, ph = (n / Cfg::kExps) & 1;
            if (!tree_wait2(&exps_full[em], ph, &exps_full[Cfg::kExps + em], ph, P.wait_limit)) ok = false;
            tree_apart<Cfg::kSpreadK, Cfg::kSpreadV, WIN>(P, sbuf, smem + Cfg::exps_off + em * 256 + hf * 64, e,
                                                          t.L - key0, P.parents ? bits : nullptr,
                                                          WIN ? prefix + qi : qi, WIN ? key0 : key0 - prefix, &own);
            F = 1.f;
            ev = unscale = 0.f;
            __syncwarp();
          }
          float x[64];
          tmem_ld32(sbuf, x);
          tmem_ld32(sbuf + 32, x + 32);
          // (WIN: whether the warp's own rows see unlike keys)
          const bool edge = WIN ? key0 + 63 > pw0 || (pw1 - key0 >= P.window && key0 + 64 > P.sinks)
                                : edge_at(t, prefix, key0, 64);
          tmem_wait_ld();
          if (edge) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              const uint32_t see = WIN ? window_bits(P, prefix + qi, key0 + 32 * w)
                                       : tree_attends(P.parents ? bits : nullptr, qi, key0 + 32 * w - prefix);
#pragma unroll
              for (int k = 0; k < 32; ++k) x[32 * w + k] = see >> k & 1 ? x[32 * w + k] : -INFINITY;
            }
          }
          float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int k = 4; k < 64; k += 2) mx[k / 2 & 3] = max3(mx[k / 2 & 3], x[k], x[k + 1]);
          const float top = fmaf(max3(mx[0], mx[1], fmaxf(mx[2], mx[3])), F, ev);
          // move the reference only when a score passes it by more than 2^8
          const bool grow = top > m_ref + (kTcRescaleThreshold + Cfg::kLift);
          float alpha = 1.f;
          if (grow) {
            alpha = ex2(m_ref - (top - Cfg::kLift));  // 0 on the first job that the row sees keys of
            m_ref = top - Cfg::kLift;
            l *= alpha;
          }
          const float add = ev - (m_ref == -INFINITY ? 0.f : m_ref);
          float2 sum = make_float2(0.f, 0.f);
          const float2 f2 = make_float2(F, F), add2 = make_float2(add, add);
          __syncwarp();  // (tcgen05.ld and .st want the warp converged)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            uint32_t pk[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              float2 e = fma_pair(make_float2(x[32 * w + 2 * k], x[32 * w + 2 * k + 1]), f2, add2);
              e = make_float2(ex2(e.x), ex2(e.y));
              sum = add_pair(sum, e);
              pk[k] = pack_half2(e.x, e.y);
            }
            tmem_st16u(sbuf + w * 16, pk);  // over scores that are in registers
          }
          l = fmaf(sum.x + sum.y, unscale, l);
          if (Q8 && ((e.x | e.y) & 256) && m_ref != -INFINITY) l = fmaf(own.y, ex2(own.x - m_ref), l);
          if (m > 0 && __any_sync(FULL, grow)) {
            // O as the chain's job before left it
            const int nb = QT == 2 && hf ? n : n - 1, yb = QT == 2 ? hf ^ 1 : nb & 1;
            if (!tree_wait(&pv_done[2 * g + yb], phase_of(nb), P.wait_limit)) ok = false;
            tc_fence_after();
            const uint32_t o_mine = uni(tmem_o + g * 128 + lane_base);
#pragma unroll 1
            for (int cc = 0; cc < HD / 32; ++cc) {
              float o[32];
              tmem_ld32(o_mine + cc * 32, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] *= alpha;
              tmem_st32(o_mine + cc * 32, o);
            }
          }
          __syncwarp();
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * g + y]);
      }

      // ---- the end of the row tile
      float w[2] = {1.f, 0.f}, M = m_ref, sum = l;  // weights of O_0 and O_1 (QT = 2: of its own)
      if constexpr (QT == 1 || Cfg::kShare) {
        float2* st = stat + (tile & 1) * 256;
        st[g * 128 + m_lane] = make_float2(m_ref, l);
      }
      if (!tree_wait(&tile_full[heard % Cfg::kAhead], (heard / Cfg::kAhead) & 1, P.wait_limit)) ok = false;
      alive = !tree_softmax_bar(!ok);
      if (Cfg::kShare && lane == 0) mbar_arrive(&stat_full[tile & 1]);
      __syncwarp();
      if constexpr (QT == 1) {
        const float2* st = stat + (tile & 1) * 256;
        const float2 a = st[m_lane], b = st[128 + m_lane];
        M = fmaxf(a.x, b.x);
        const float ref = M == -INFINITY ? 0.f : M;
        w[0] = ex2(a.x - ref);
        w[1] = ex2(b.x - ref);
        sum = a.y * w[0] + b.y * w[1];
      }
      if (tiles > 0) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if ((QT == 1 || k == g) && ok && !tree_wait(&o_full[k], oc & 1, P.wait_limit)) ok = false;
        ++oc;
      }
      tc_fence_after();
      const bool whole = t.slot < 0;
      const float inv = whole ? 1.f / sum : 1.f;
      const uint32_t* bad = bad_s + (tile % Cfg::kBad) * kTreeWords;
      // (kShare: of the first half of the columns)
      constexpr int kCols = (QT == 1 ? HD / 2 : HD) / (Cfg::kShare ? 2 : 1);
      const int col0 = QT == 1 ? g * kCols : 0, cols = kCols;
      bool any_bad = false;
      if constexpr (Cfg::kLook) {
        any_bad = bad[0] != 0;
      } else if (drafts) {
        uint32_t hit = 0;
#pragma unroll
        for (int k = 0; k < kTreeWords; ++k) hit |= bad[k];
        any_bad = tree_softmax_bar(hit != 0);
      }
      const bool swap = WIN && whole;
      __half* dst4[4];
      if (swap) rows_out(row_ok ? P.out + (tok * P.num_heads + t.kvh * G + head) * HD : nullptr, dst4);
#pragma unroll 1
      for (int cc = 0; swap && cc < cols / 32; ++cc) {
        float o[32];
        __syncwarp();
        const uint32_t from = uni(tmem_o + (QT == 2 ? g * 128 : 0) + col0 + cc * 32 + lane_base);
#pragma unroll
        for (int half = 0; half < 32; half += 16) {
          float x[16];
          tmem_ld<16>(from + half, o + half);
          if (QT == 1) tmem_ld<16>(from + half + 128, x);
          tmem_wait_ld();
          if constexpr (QT == 1) {
#pragma unroll
            for (int k = 0; k < 16; ++k)
              o[half + k] = (w[0] > 0.f ? o[half + k] * w[0] : 0.f) + (w[1] > 0.f ? x[k] * w[1] : 0.f);
          }
        }
        if (cc + 1 == cols / 32) {  // both O (QT = 2: the chain's own) are read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(QT == 2 && g ? o_free1 : o_free);
        }
        uint32_t h[4][4];
        pack32(o, inv, h);
        if (ok) store32(h, dst4, col0 + cc * 32);
      }
#pragma unroll 1
      for (int cc = 0; !swap && cc < cols / 16; ++cc) {
        const int d0 = col0 + cc * 16;
        float o[16], x[16];
        __syncwarp();  // rows that there are not have left the rest of the loop out
        const uint32_t from = uni(tmem_o + (QT == 2 ? g * 128 : 0) + d0 + lane_base);
        if (tiles > 0) tmem_ld<16>(from, o);
        if (QT == 1 && tiles > 0) tmem_ld<16>(from + 128, x);
        tmem_wait_ld();
        if (cc + 1 == cols / 16) {  // both O are read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(WIN && QT == 2 && g ? o_free1 : o_free);
        }
        if (!row_ok || !ok) continue;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          // (weight 0: a chain none of whose keys this row saw)
          const float v = QT == 2 ? o[k] : (w[0] > 0.f ? o[k] * w[0] : 0.f) + (w[1] > 0.f ? x[k] * w[1] : 0.f);
          o[k] = tiles > 0 ? v : 0.f;
        }
        if (whole) {
          uint4* dst = reinterpret_cast<uint4*>(P.out + (tok * P.num_heads + t.kvh * G + head) * HD + d0);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            dst[k] = make_uint4(pack_half2(o[8 * k] * inv, o[8 * k + 1] * inv),
                                pack_half2(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                                pack_half2(o[8 * k + 4] * inv, o[8 * k + 5] * inv),
                                pack_half2(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
        } else {
          float* dst = S.part_o + (int64_t(t.slot) * HD + d0) * Cfg::kRows + tr;  // by columns
#pragma unroll
          for (int k = 0; k < 16; ++k) dst[k * Cfg::kRows] = o[k];
        }
      }
      if (!whole && row_ok && (QT == 2 || g == 0))
        S.part_ml[int64_t(t.slot) * Cfg::kRows + tr] = make_float2(M, sum);
      if (any_bad) {
        __syncwarp();  // (WIN: a row's results are stored by four lanes)
        if (row_ok && alive) {
          __half* to = whole ? P.out + (tok * P.num_heads + t.kvh * G + head) * HD : nullptr;
          float* part = S.part_o + int64_t(max(t.slot, 0)) * HD * Cfg::kRows + tr;
          if constexpr (WIN)
            window_patch<Q8, TOK, 64>(P, told[(heard - 1) % Cfg::kAhead], prefix + qi, to, part, Cfg::kRows, col0, 1,
                                  col0 + cols);
          else
            tree_patch<Q8>(P, t.b, t.q, prefix, t.kvh, qi, bad, P.parents ? bits : nullptr, t.s0 * TOK, t.s1 * TOK, to,
                           part, Cfg::kRows, col0, 1, col0 + cols);
        }
        if constexpr (!Cfg::kLook) {  // (the looking warps clear their flags themselves)
          tree_softmax_bar();
          if (tid - 128 < kTreeWords) bad_s[(tile % Cfg::kBad) * kTreeWords + tid - 128] = 0;
        }
      }
      if constexpr (SEG) {
        const int seg = told[(heard - 1) % Cfg::kAhead].seg;
        if (seg && row_ok && ok)
          tree_fold<HD, Cfg::kRows, 1>(S, worker, seg, QT == 1 ? g : 0, tr, make_float2(M, sum), tr, Cfg::kRows,
                                       P.out + (tok * P.num_heads + t.kvh * G + head) * HD, col0, col0 + cols);
      }
      n0 += tiles;
      ++tile;
    }
  } else if (warp >= 12) {
    if constexpr (Cfg::kLook) {
      // ================= V tiles looked through before their products; rows written out =================
      // The first V tile of the next row tile is looked through before a row tile's rows are written: its
      // product waits for both.
      const int quarter = warp & 3, m_lane = quarter * 32 + lane;
      const uint32_t lane_base = uint32_t(quarter * 32) << 16;
      const float2* stat = reinterpret_cast<const float2*>(smem + Cfg::stat_off);
      int tile = 0, vslot = 0, vphase = 0, oc = 0;
      auto look = [&](const Tile& t, int p0, int i) {
        if (!tree_wait(&vfull[vslot], vphase, P.wait_limit)) {
          ok = false;
          return;
        }
#pragma unroll 1
        for (int hf = 0; hf < 2; ++hf) {
          const int key0 = key_of(t, t.s0 + i, hf);
          if (edge_at(t, p0, key0, 64))
            clean_v_window<H2>(vring + vslot * Cfg::kTile, t, p0, P.sinks, hf * 64, key0,
                               bad_s + (tile % Cfg::kBad) * kTreeWords, tid - 384);
        }
        if (lane == 0) mbar_arrive(&vready[vslot]);
        __syncwarp();
        if (++vslot == VS) {
          vslot = 0;
          vphase ^= 1;
        }
      };
      auto write_out = [&](const Tile& t, int k) {
        const float2* st = stat + (k & 1) * 256;
        const bool whole = t.slot < 0;
        if (!tree_wait(&stat_full[k & 1], (k >> 1) & 1, P.wait_limit)) {
          ok = false;
          return;
        }
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
          const int tr = x * 128 + m_lane, qi = token_of(t, tr);
          const int64_t tok = int64_t(t.q_start) + qi;
          const bool row_ok = qi < t.q && tok < P.tokens;
          const float inv = whole ? 1.f / st[tr].y : 1.f;
          __half* mine = row_ok ? P.out + (tok * P.num_heads + t.kvh * G + head_of(t, tr, qi)) * HD : nullptr;
          __half* dst[4];
          rows_out(mine, dst);
          float* part = S.part_o + int64_t(max(t.slot, 0)) * HD * Cfg::kRows + tr;  // by columns
          if (!tree_wait(&o_full[x], oc & 1, P.wait_limit)) {
            ok = false;
            return;
          }
          tc_fence_after();
          float o[2][32];
          __syncwarp();
          const uint32_t from = uni(tmem_o + x * 128 + HD / 2 + lane_base);
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) tmem_ld32(from + cc * 32, o[cc]);
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(x ? o_free1 : o_free);
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            if (whole) {
              uint32_t h[4][4];
              pack32(o[cc], inv, h);
              store32(h, dst, HD / 2 + cc * 32);
            } else if (row_ok) {
#pragma unroll
              for (int j = 0; j < 32; ++j) part[int64_t(HD / 2 + cc * 32 + j) * Cfg::kRows] = o[cc][j];
            }
          }
          if (bad_s[(k % Cfg::kBad) * kTreeWords]) {
            __syncwarp();
            if (row_ok)
              window_patch<Q8, TOK, 64>(P, t, t.L - t.q + qi, whole ? mine : nullptr, part, Cfg::kRows, HD / 2, 1, HD);
            __syncwarp();
          }
          if constexpr (SEG) if (t.seg && row_ok)
            tree_fold<HD, Cfg::kRows, 1>(S, worker, t.seg, 1, tr, st[tr], tr, Cfg::kRows, mine, HD / 2, HD);
        }
        ++oc;
      };
      Tile t;
      bool have = next_tile(t);
      int p0 = have ? t.first() : 0;  // (no tile told, t is nothing)
      if (have) look(t, p0, 0);
      while (ok && have) {
        // the flags of four row tiles ago, which every warp has written out
        if (warp == 12 && lane == 0) bad_s[((tile + 4) % Cfg::kBad) * kTreeWords] = 0;
        const int tiles = key_tiles(t);
        for (int i = 1; i < tiles && ok; ++i) look(t, p0, i);
        if (!ok) break;
        const Tile done = t;
        ++tile;
        have = next_tile(t);
        p0 = have ? t.first() : 0;
        if (have) look(t, p0, 0);
        if (Cfg::kShare && ok) write_out(done, tile - 1);
      }
    }
    if constexpr (Q8) {
    // ================= codes to fp16 operands =================
    const int part = (warp - 12) / Cfg::kConv, sub = (warp - 12) % Cfg::kConv, kv = part >> 1;
    constexpr int ROWS = 64 / Cfg::kConv;  // of this warp
    constexpr int CH = HD / 8;             // 8-code chunks of a row: 16 bytes of operand
    constexpr int RPI = 32 / CH;           // rows that the warp takes at a time
    const int ch = lane % CH, row0 = (part & 1) * 64 + sub * ROWS + lane / CH;  // this lane's first row
    uint64_t* full = kv ? vfull : kfull;
    uint64_t* empty = kv ? vempty : kempty;
    uint64_t* landed = sfull + (kv ? 2 * Cfg::kKRounds : 0) + (part & 1);  // [2 * round]
    const int rounds = kv ? Cfg::kVRounds : Cfg::kKRounds;
    uint64_t* taken = sempty + (kv ? Cfg::kKStages : 0);
    uint8_t* stage = smem + Cfg::stage_off + (kv ? Cfg::kKStages : 0) * Cfg::kStageBytes + sub * ROWS * HD + lane * 8;
    // this lane's places in the operand: the 64-dim half ch / 8 of row0, row0 + RPI, ...
    uint8_t* operand = (kv ? vring : kring) + (ch >> 3) * Cfg::kHalf + row0 * 128;
    // (rings of this warp's tile: slots and phases counted, as a remainder takes long)
    const int ns = kv ? VS : KS, nst = kv ? Cfg::kVStages : Cfg::kKStages;
    int slot = 0, phase = 0, st = part & 1, round = 0, lphase = 0, em = 0, ephase = 0, mm = 0, tile = 0;
    Tile t;
    // The largest exponent of the tile in slot `es`, unit u of the row tile, of the rows that are the context's
    // (WIN: attended by some row); of each kind the first part's warp tells the softmax, and whether
    // some lie far below it.
    auto look = [&](int u, int es, int ph, int m, int& top) {
      if (!tree_wait(&exps_full[kv * Cfg::kExps + es], ph, P.wait_limit)) return false;
      const uint32_t e4 = *reinterpret_cast<const uint32_t*>(smem + Cfg::exps_off + es * 256 + kv * 128 + lane * 4);
      // this lane's four (of trees not by key_of: the halves' own sums took trees of 16 from 92.5 to 94.6 us)
      const int key0 = WIN ? key_of(t, u, lane >> 4) + (lane & 15) * 4 : u * TOK + lane * 4, left = t.L - key0;
      // (WIN: the keys between the sinks and the first row's window are nobody's)
      int behind = 0;
      uint32_t gap = 0;
      if constexpr (WIN) {
        behind = key0 - P.sinks;
        gap = uint32_t(max(t.lo - P.sinks, 0));
      }
      int low = 255;
      top = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int e = int(e4 >> (8 * j) & 255);
        const bool in = left > j && uint32_t(behind + j) >= gap;
        top = max(top, in ? e : 0);
        low = min(low, in ? e : 255);
      }
      top = max(__reduce_max_sync(FULL, top), kExpLeastByte);
      low = __reduce_min_sync(FULL, low);
      if ((part & 1) == 0 && sub == 0 && lane == 0) {
        reinterpret_cast<int*>(&meta[m])[kv] = top | (top - low > (kv ? Cfg::kSpreadV : Cfg::kSpreadK) ? 256 : 0);
        mbar_arrive(&meta_full[m]);
      }
      return true;
    };
    while (ok && next_tile(t)) {
      const int tiles = key_tiles(t), prefix = t.L - t.q;
      int p0 = prefix;
      if constexpr (WIN) p0 = t.first();
      int top = 0;
      if (tiles > 0 && !look(t.s0, em, ephase, mm, top)) {
        ok = false;
        break;
      }
      for (int i = 0; i < tiles; ++i) {
        // of row 0, as this part counts
        const int key0 = WIN ? key_of(t, t.s0 + i, part & 1) - (part & 1) * 64 : (t.s0 + i) * TOK;
        uint8_t* exps = smem + Cfg::exps_off + em * 256 + kv * 128;
        if (!tree_wait(&landed[2 * round], lphase, P.wait_limit)) {
          ok = false;
          break;
        }
        uint8_t* src = stage + st * Cfg::kStageBytes;
        uint8_t* dst = operand + slot * Cfg::kTile;
        if (!WIN && edge_at(t, p0, key0, TOK)) {
          // the tile reaches the drafts: rows behind the context become 0, and
          // non-finite elements of the drafts' V rows leave the product
#pragma unroll 1
          for (int k = 0; k < ROWS / RPI; ++k) {
            const int key = key0 + row0 + k * RPI, a = key - prefix;
            uint2* p = reinterpret_cast<uint2*>(src + k * 256);
            uint2 x = *p;
            bool hit = key >= t.L;
            if (hit) {
              x = make_uint2(0, 0);
              if (ch == 0) exps[row0 + k * RPI] = uint8_t(top);
            } else if (kv && key >= prefix) {
              hit = clear_nonfinite<true>(x.x);
              hit |= clear_nonfinite<true>(x.y);
              if (hit) atomicOr(&bad_s[(tile % Cfg::kBad) * kTreeWords + (a >> 5) % kTreeWords], 1u << (a & 31));
            }
            if (hit) *p = x;
          }
          __syncwarp();
        }
        if constexpr (WIN) if (edge_at(t, p0, key0 + (part & 1) * 64, 64)) {
          // An end of the windows: rows that no row of the tile attends become 0, whatever their exponents, and
          // non-finite elements of the V rows that not every row sees leave the product. By ranges of
          // rows (a look at every row took 2.5 us).
          uint8_t* rows = src - lane * 8;
          const auto row = [&](int key) { return min(max(key - (key0 + (part & 1) * 64), 0), 64) * HD; };
#pragma unroll 1
          for (int upper = 0; upper < 2; ++upper) {
            const int end = upper ? 64 * HD : row(t.lo);
            for (int at = row(upper ? t.L : P.sinks) + lane * 16; at < end; at += 512)
              *reinterpret_cast<uint4*>(rows + at) = make_uint4(0, 0, 0, 0);
            const int last = kv ? row(upper ? t.L : min(t.lo1, p0 + 1)) : 0;
#pragma unroll 1
            for (int at = row(upper ? p0 + 1 : max(t.lo, P.sinks)) + lane * 16; at < last; at += 512) {
              uint4 v = lds128(rows + at);
              if (!(nan_codes(v.x) | nan_codes(v.y) | nan_codes(v.z) | nan_codes(v.w))) continue;
              clear_nonfinite<true>(v.x);
              clear_nonfinite<true>(v.y);
              clear_nonfinite<true>(v.z);
              clear_nonfinite<true>(v.w);
              *reinterpret_cast<uint4*>(rows + at) = v;
              atomicOr(&bad_s[(tile % Cfg::kBad) * kTreeWords], 1u);
            }
          }
          __syncwarp();
        }
        // all of the part into registers, so that its stage is free for the next copy
        // while it is widened
        uint2 x[ROWS / RPI];
#pragma unroll
        for (int k = 0; k < ROWS / RPI; ++k) x[k] = *reinterpret_cast<const uint2*>(src + k * 256);
        // The stage's next copy comes by another proxy, so it does not queue behind these loads (nor
        // behind the stores above) as an ordinary store would: without the fence their last
        // rows were at times the next copy's, where the softmax warps' stores at the end of a
        // row tile held the loads up.
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&taken[st]);
        // factors of the rows lane, lane + 32 of this warp: 2^-diff, as far down as goes
        uint32_t fac[ROWS / 32];
#pragma unroll
        for (int k = 0; k < ROWS / 32; ++k) {
          const uint32_t diff = uint32_t(top) - exps[(part & 1) * 64 + sub * ROWS + 32 * k + lane];
          fac[k] = (15u - min(diff, uint32_t(kv ? Cfg::kSpreadV : Cfg::kSpreadK))) * 0x04000400u;
        }
        if (!tree_wait(&empty[slot], phase ^ 1, P.wait_limit)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int k = 0; k < ROWS / RPI; ++k) {
          const int rr = k * RPI;
          const uint32_t f = __shfl_sync(FULL, fac[rr / 32], (rr & 31) + lane / CH);
          *reinterpret_cast<uint4*>(dst + rr * 128 + (((ch & 7) ^ ((row0 + rr) & 7)) << 4)) =
              make_uint4(hmul2u(e4m3x2_half2(x[k].x), f), hmul2u(e4m3x2_half2(x[k].x >> 16), f),
                         hmul2u(e4m3x2_half2(x[k].y), f), hmul2u(e4m3x2_half2(x[k].y >> 16), f));
        }
        mm = (mm + 1) % Cfg::kMeta;
        if (++em == Cfg::kExps) {
          em = 0;
          ephase ^= 1;
        }
        // the next tile's exponents now, or its softmax would wait for them (trees of 16: 93.8 us so, 103
        // at the tile's own turn, 98 before the wait for the place, 97 behind the hand-over)
        if (i + 1 < tiles && !look(t.s0 + i + 1, em, ephase, mm, top)) {
          ok = false;
          break;
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[slot]);
        if (++slot == ns) {
          slot = 0;
          phase ^= 1;
        }
        if ((st += 2) >= nst) st -= nst;
        if (++round == rounds) {
          round = 0;
          lphase ^= 1;
        }
      }
      ++tile;
    }
    }
  }
  if (!ok && lane == 0) set_status(P.status, PA_STATUS_BIT_TIMEOUT);
  // ---- teardown: every tcgen05 op has completed before TMEM is freed
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tree_wait(all_done, 0);
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
}

// Launches the kernel of a tile shape and its combine pass; with `need`, only
// says how much workspace they take. (long: called by the others, for tiles in segments)
cudaError_t tree_tc(const TreeParams& P, int head_size, bool q8, int64_t rows, int sms, size_t* need,
                    void* ws, cudaStream_t s);
cudaError_t window_tc(const TreeParams& P, int head_size, bool q8, int64_t rows, int sms, size_t* need,
                      void* ws, cudaStream_t s);
cudaError_t tree_tc_long(const TreeParams& P, int head_size, bool q8, int64_t rows, int sms, size_t* need,
                         void* ws, cudaStream_t s);
cudaError_t window_tc_long(const TreeParams& P, int head_size, bool q8, int64_t rows, int sms, size_t* need,
                           void* ws, cudaStream_t s);

}  // namespace pa
