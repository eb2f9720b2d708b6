// Tree attention on the warp-level tensor instructions, for up to 32 rows (a
// group of heads times a few drafts) per tile and K and V heads of 64, 128 or 256
// dims, over the fp16 or the 8-bit cache.
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
// Every warp streams its keys through a ring of its own with cp.async, so there
// is no block-wide barrier between the ends of a tile.
#pragma once

#include "pa_decode_mma.cuh"
#include "pa_tree_split.cuh"

namespace pa {

template <int HD, bool Q8, int NT>
struct TreeMma {
  static constexpr int kWarps = 4;
  static constexpr int kRowBytes = HD * (Q8 ? 1 : 2);
  static constexpr int kChunks = kRowBytes / 16;            // 16-byte chunks of a row
  static constexpr int kElems = Q8 ? 16 : 8;                // elements of a chunk
  static constexpr int kSub = kRowBytes <= 128 ? 32 : 16;   // keys a warp takes at a time
  static constexpr int kMT = kSub / 16;
  static constexpr int kRows = 8 * NT;
  static constexpr uint32_t kV = kSub * kRowBytes;          // V behind K in a stage
  static constexpr uint32_t kExps = 2 * kV;                 // then 2 x kSub exponent bytes
  static constexpr uint32_t kStage = 2 * kV + (Q8 ? 64 : 0);
  static constexpr int kCtas = kStage > 9000 ? 1 : 2;       // CTAs of an SM
  static constexpr int kStages = HD == 64 && Q8 ? 5 : 3;
  static constexpr uint32_t kRing = kWarps * kStages * kStage;
  static constexpr int kMergeStride = HD + 4;               // floats of a merge row
  static constexpr uint32_t kMerge = kWarps * kRows * (kMergeStride + 2) * 4;
  static_assert(kMerge <= kRing, "the merge reuses the ring");
  static constexpr uint32_t q_off = kRing;
  static constexpr uint32_t mask_off = q_off + kRows * HD * 2;
  static constexpr uint32_t bad_off = mask_off + kRows * kTreeWords * 4;
  static constexpr uint32_t bytes = bad_off + kTreeWords * 4;
  static_assert(bytes * kCtas + 1024 * kCtas <= 227 * 1024 + 1024, "shared memory");
};

// The chunk's place in its row: rows of a line or more spread over all banks.
template <int CHUNKS>
__device__ __forceinline__ int tree_swz(int chunk, int row) {
  return CHUNKS >= 8 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
  const uint32_t n = ok ? 16 : 0;  // 0: the 16 bytes are zeroed
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
    tree_mma_kernel(const TreeParams P, const TreeSplit S) {
  using Cfg = TreeMma<HD, Q8, NT>;
  using Line = TreeLine<Cfg::kSub, Cfg::kRows>;
  constexpr int SUB = Cfg::kSub, MT = Cfg::kMT, NR = Cfg::kRows, NW = Cfg::kWarps;
  constexpr int RB = Cfg::kRowBytes, C = Cfg::kChunks, E = Cfg::kElems;
  constexpr int OT = HD / 16;  // m-tiles of O^T
  constexpr unsigned FULL = 0xffffffffu;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  uint8_t* ring = smem + warp * (Cfg::kStages * Cfg::kStage);
  uint8_t* q_s = smem + Cfg::q_off;
  uint32_t* mask_s = reinterpret_cast<uint32_t*>(smem + Cfg::mask_off);
  uint32_t* bad_s = reinterpret_cast<uint32_t*>(smem + Cfg::bad_off);

  const int64_t total = Line::total(P, lane);
  const int nact = Line::ctas(total, int(gridDim.x), S.min_units);
  if (int(blockIdx.x) >= nact) return;
  const int64_t u0 = Line::begin(total, blockIdx.x, nact), u1 = Line::begin(total, blockIdx.x + 1, nact);
  if (u0 >= u1) return;
  int64_t before;
  int q_start;
  int b = Line::find(P, u0, lane, before, q_start);
  if (b < 0) return;
  typename Line::Seq seq = Line::load(P, b);
  const int G = P.group, bs = P.block_size;
  const int64_t row_stride = int64_t(P.kv_heads) * RB;

  for (int64_t u = u0; u < u1;) {
    while (u >= before + seq.total(P)) {
      before += seq.total(P);
      q_start += seq.q;
      seq = Line::load(P, ++b);
    }
    const int tile = int((u - before) / seq.units);
    const int s0 = int((u - before) % seq.units);
    const int s1 = int(min(int64_t(seq.units), s0 + (u1 - u)));
    const int kvh = tile / seq.tiles, r0 = (tile % seq.tiles) * NR;
    const int L = seq.L, prefix = L - seq.q;
    const bool drafts = s1 * SUB > prefix;  // the keys reach the current tokens
    const int nmine = s1 - s0 > warp ? (s1 - s0 - warp + NW - 1) / NW : 0;

    // ---- the keys' stream. Lane l holds the blocks of 16 keys each that the
    // units to come need: MT a unit, 32 / MT units a window, and the next window's.
    const int32_t* table = P.block_tables + int64_t(b) * P.max_blocks_per_seq;
    constexpr int WIN = 32 / MT;
    auto blocks_of = [&](int n0) {
      const int n = n0 + lane / MT;
      const int key = (s0 + warp + n * NW) * SUB + (lane % MT) * 16;
      return n < nmine && key < L ? table[key / bs] : 0;
    };
    int win0 = 0, cur = blocks_of(0), next = blocks_of(WIN);
    auto issue = [&](int n) {
      if (n < nmine) {
        if (n >= win0 + WIN) {
          win0 += WIN;
          cur = next;
          next = blocks_of(win0 + WIN);
        }
        const uint32_t dst = smem_u32(ring + (n % Cfg::kStages) * Cfg::kStage);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const int block = __shfl_sync(FULL, cur, (n - win0) * MT + m);
          const int key = (s0 + warp + n * NW) * SUB + m * 16;
          const bool ok = block >= 0 && block < P.num_blocks;
          if (!ok && lane == 0) set_status(P.status, PA_STATUS_BIT_BLOCK_INDEX);
          const int place = key % bs;
          const int64_t base = ok && key < L ? (int64_t(block) * bs + place) * row_stride + int64_t(kvh) * RB : 0;
#pragma unroll
          for (int k = 0; k < C / 2; ++k) {
            const int at = lane + 32 * k, row = at / C, ch = at % C;
            const bool in = ok && key + row < L;
            const int64_t off = in ? base + row * row_stride + ch * 16 : 0;
            const uint32_t to = dst + (m * 16 + row) * RB + tree_swz<C>(ch, row) * 16;
            cp_async16(to, P.key_cache + off, in);
            cp_async16(to + Cfg::kV, P.value_cache + off, in);
          }
          if constexpr (Q8) {
            if (lane < 2) {
              const bool in = ok && key < L;
              const int64_t off = in ? (int64_t(block) * P.kv_heads + kvh) * bs + place : 0;
              cp_async16(dst + Cfg::kExps + lane * 32 + m * 16, (lane ? P.value_exps : P.key_exps) + off, in);
            }
          }
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int n = 0; n < Cfg::kStages; ++n) issue(n);

    // ---- the query tile as B fragments, and what its rows see of the drafts
    for (int at = tid; at < NT * OT * 32; at += NW * 32) {
      const int nt = at / (OT * 32), ks = at / 32 % OT, l = at % 32;
      const int r = r0 + nt * 8 + (l >> 2), i = r / G;
      const int s = ks / (E / 4), j = ks % (E / 4), lc = l & 3;
      const int ch = C >= 8 ? 2 * lc + (s & 1) + 8 * (s >> 1) : lc;
      const int64_t t = int64_t(q_start) + i;
      uint2 v = make_uint2(0, 0);
      if (i < seq.q && t < P.tokens)
        v = *reinterpret_cast<const uint2*>(P.query + (t * P.num_heads + kvh * G + r % G) * HD + ch * E + 4 * j);
      *reinterpret_cast<uint2*>(q_s + at * 8) = v;
    }
    if (tid < kTreeWords) bad_s[tid] = 0;
    if (drafts && tid < NR) {
      uint32_t bits[kTreeWords];
#pragma unroll
      for (int w = 0; w < kTreeWords; ++w) bits[w] = 0;
      const int i = (r0 + tid) / G;
      if (P.parents && i < seq.q && int64_t(q_start) + i < P.tokens)
        tree_ancestors(P, P.parents + q_start, i, bits);
#pragma unroll
      for (int w = 0; w < kTreeWords; ++w) mask_s[tid * kTreeWords + w] = bits[w];
    }
    int token[NT][2];  // of this lane's rows nt * 8 + 2 c + e
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) token[nt][e] = (r0 + nt * 8 + 2 * c + e) / G;
    auto sees = [&](int row, int i, int a) {  // draft a from a row of draft i
      return P.parents ? (mask_s[row * kTreeWords + (a >> 5)] >> (a & 31) & 1u) != 0 : a <= i;
    };
    __syncthreads();

    float m_run[NT][2], l_run[NT][2], o[OT][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m_run[nt][0] = m_run[nt][1] = -INFINITY;
      l_run[nt][0] = l_run[nt][1] = 0.f;
#pragma unroll
      for (int k = 0; k < OT; ++k) o[k][nt][0] = o[k][nt][1] = o[k][nt][2] = o[k][nt][3] = 0.f;
    }

    for (int n = 0; n < nmine; ++n) {
      cp_async_wait<Cfg::kStages - 1>();
      __syncwarp();
      uint8_t* kb = ring + (n % Cfg::kStages) * Cfg::kStage;
      uint8_t* vb = kb + Cfg::kV;
      const int j0 = (s0 + warp + n * NW) * SUB;
      const bool edge = j0 + SUB > prefix;

      // ---- S^T = K . Q^T
      float s[MT][NT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[mt][nt][0] = s[mt][nt][1] = s[mt][nt][2] = s[mt][nt][3] = 0.f;
        const uint8_t* row = kb + (mt * 16 + g) * RB;
#pragma unroll
        for (int sc = 0; sc < C / 4; ++sc) {
          const int ch = tree_swz<C>(C >= 8 ? 2 * c + (sc & 1) + 8 * (sc >> 1) : c, g);
          const uint4 xa = lds128(row + ch * 16), xb = lds128(row + 8 * RB + ch * 16);
          const uint32_t* wa = reinterpret_cast<const uint32_t*>(&xa);
          const uint32_t* wb = reinterpret_cast<const uint32_t*>(&xb);
#pragma unroll
          for (int j = 0; j < E / 4; ++j) {
            uint32_t a[4];
            if constexpr (Q8) {
              a[0] = e4m3x2_half2(wa[j]);
              a[1] = e4m3x2_half2(wb[j]);
              a[2] = e4m3x2_half2(wa[j] >> 16);
              a[3] = e4m3x2_half2(wb[j] >> 16);
            } else {
              a[0] = wa[2 * j];
              a[1] = wb[2 * j];
              a[2] = wa[2 * j + 1];
              a[3] = wb[2 * j + 1];
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint2 q = *reinterpret_cast<const uint2*>(q_s + ((nt * OT + sc * (E / 4) + j) * 32 + lane) * 8);
              mma_16816(s[mt][nt], a, q.x, q.y);
            }
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
            int ke = kb[Cfg::kExps + kk], ve = kb[Cfg::kExps + 32 + kk];
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
              if (edge) {
                const bool in = key < prefix || (key < L && sees(nt * 8 + 2 * c + e, token[nt][e], key - prefix));
                if (!in) x = -INFINITY;
              }
            }
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
        // non-finite elements of the drafts' V rows leave the product
        for (int at = lane; at < SUB * C; at += 32) {
          const int row = at / C, key = j0 + row;
          if (key < prefix || key >= L) continue;
          uint4* p = reinterpret_cast<uint4*>(vb + row * RB + (at % C) * 16);
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
        const uint8_t* v0 = vb + (mt * 16 + 2 * c) * RB;
        if constexpr (C >= 8) {
#pragma unroll
          for (int uu = 0; uu < C / 8; ++uu) {
            const int even = ((g + 8 * uu) ^ (2 * c)) * 16, odd = ((g + 8 * uu) ^ (2 * c + 1)) * 16;
            const uint4 x0 = lds128(v0 + even), x1 = lds128(v0 + RB + odd);
            const uint4 x2 = lds128(v0 + 8 * RB + even), x3 = lds128(v0 + 9 * RB + odd);
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
            x[k] = *reinterpret_cast<const uint2*>(vb + (mt * 16 + row) * RB + tree_swz<C>(g >> 1, row) * 16 + (g & 1) * 8);
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
      __syncwarp();
      issue(n + Cfg::kStages);
    }
    cp_async_wait<0>();
    if (u1 - u <= s1 - s0) launch_dependents();  // this CTA's last tile

    // ---- the warps' states into shared memory, and merged
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
    __syncthreads();  // every warp is done with its ring
    float* o_s = reinterpret_cast<float*>(smem);
    float2* ml_s = reinterpret_cast<float2*>(o_s + NW * NR * Cfg::kMergeStride);
    constexpr int DL = HD / 8;  // dims of a lane's share, in runs of min(E, DL)
    constexpr int RUN = E < DL ? E : DL;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int n = nt * 8 + 2 * c + e;
        if (g == 0) ml_s[warp * NR + n] = make_float2(m_run[nt][e], l_run[nt][e]);
        float* row = o_s + (warp * NR + n) * Cfg::kMergeStride;
#pragma unroll
        for (int k = 0; k < OT; ++k) {
          const int run = 2 * k / RUN, d = (g + 8 * run) * RUN + 2 * k % RUN;
          *reinterpret_cast<float2*>(row + d) = make_float2(o[k][nt][e], o[k][nt][2 + e]);
        }
      }
    __syncthreads();
    const bool whole = s0 == 0 && s1 == seq.units;
    const int slot = 2 * int(blockIdx.x) + (u == u0 ? 0 : 1);
    for (int at = tid; at < NR * (HD / 2); at += NW * 32) {
      const int n = at / (HD / 2), d = at % (HD / 2) * 2;
      const int r = r0 + n, i = r / G;
      const int64_t t = int64_t(q_start) + i;
      if (i >= seq.q || t >= P.tokens) continue;
      float M = ml_s[n].x;
#pragma unroll
      for (int w = 1; w < NW; ++w) M = fmaxf(M, ml_s[w * NR + n].x);
      const float ref = M == -INFINITY ? 0.f : M;
      float sum = 0.f, x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float2 ml = ml_s[w * NR + n];
        const float f = ex2(ml.x - ref);
        const float2 v = *reinterpret_cast<const float2*>(o_s + (w * NR + n) * Cfg::kMergeStride + d);
        sum = fmaf(ml.y, f, sum);
        x = fmaf(v.x, f, x);
        y = fmaf(v.y, f, y);
      }
      if (drafts) {
        // what was taken out of the product, for the rows that see it
        for (int w = 0; w < kTreeWords; ++w) {
          if (!bad_s[w]) continue;
          for (int a = w * 32; a < seq.q; ++a) {
            if ((a >> 5) % kTreeWords != w || !(bad_s[w] >> (a & 31) & 1) || !sees(n, i, a)) continue;
            const int key = prefix + a;
            if (key < s0 * SUB || key >= s1 * SUB) continue;
            const int block = table[key / bs];
            if (block < 0 || block >= P.num_blocks) continue;
            const uint8_t* vr = P.value_cache + (int64_t(block) * bs + key % bs) * row_stride + int64_t(kvh) * RB;
            const float2 v = Q8 ? h2f2(e4m3x2_half2(*reinterpret_cast<const uint16_t*>(vr + d)))
                                : h2f2(*reinterpret_cast<const uint32_t*>(vr + 2 * d));
            if (!isfinite(v.x)) x += v.x;
            if (!isfinite(v.y)) y += v.y;
          }
        }
      }
      if (whole) {
        __half2* dst = reinterpret_cast<__half2*>(P.out + (t * P.num_heads + kvh * G + r % G) * HD + d);
        *dst = __floats2half2_rn(x / sum, y / sum);
      } else {
        const int64_t row = int64_t(slot) * NR + n;
        *reinterpret_cast<float2*>(S.part_o + row * HD + d) = make_float2(x, y);
        if (d == 0) S.part_ml[row] = make_float2(M, sum);
      }
    }
    __syncthreads();  // the ring is free again
    u += s1 - s0;
  }
}

// Launches the kernel of a tile shape and its combine pass; with `need`, only
// says how much workspace they take.
cudaError_t tree_mma_64(const TreeParams& P, bool q8, int nt, int sms, size_t* need, void* ws, cudaStream_t s);
cudaError_t tree_mma_128(const TreeParams& P, bool q8, int nt, int sms, size_t* need, void* ws, cudaStream_t s);
cudaError_t tree_mma_256(const TreeParams& P, bool q8, int nt, int sms, size_t* need, void* ws, cudaStream_t s);

}  // namespace pa
