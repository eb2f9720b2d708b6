// Norm and rotation of query and key heads, and the 8-bit cache written and
// read back (pa_cache.h).
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "pa_cache.h"
#include "pa_device.cuh"
#include "pa_e4m3.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

enum RowMode { kRotate, kWrite, kStore };

// With kRows * kBatches rows to a group of lanes where that leaves 16 warps for
// each of 152 SMs, kRows at once; with one row to it where there are fewer (one
// token of 32 + 8 heads of 128 turned: 2.0 us so, 2.6 us with two rows; 8192
// tokens: 34 us with 2 x 2, 43 us with one).
constexpr int kRows = 2;
constexpr int kBatches = 2;
constexpr int64_t kManyWarps = 152 * 16;

struct RowParams {
  const __half *query, *key, *value, *q_weight, *k_weight;
  const float* cos_sin;
  const int32_t *positions, *block_tables, *context_lens, *q_seqlens;
  __half *q_out, *k_out;
  uint8_t *key_cache, *key_exps, *value_cache, *value_exps;
  uint32_t* status;
  int64_t tokens, query_stride, key_stride, value_stride;
  int batch, heads, kv_heads, hk, hv, rot, interleaved, max_positions;
  int block_size, num_blocks, max_blocks_per_seq, max_rows;
  int lane_shift;  // log2 of the lanes of a row
  int batches;     // of rows in a warp, at most
  uint32_t q_slices, k_slices, slices;  // warps of a token: its queries', keys', all
  float eps, inv_hk;
  int axes;                                 // of the positions [axes][tokens]; 0: one, [tokens]
  uint32_t axis_of[PA_MAX_HEAD_SIZE / 32];  // the axis of each pair, two bits a pair
};

__device__ __forceinline__ void report(uint32_t* status, uint32_t bit) {
  if (status) atomicOr(status, bit);
}

// Sequence and index in it of token t: the last sequence whose tokens begin at
// or before t. Warp-collective, 128 sequences at a time; -1 past the last one.
// Every sequence counts with the length it states (a negative one with 0), whether it
// is valid or not: the rows lie as the lengths say. The sums stop at the number
// of tokens, past which no token looks.
__device__ __forceinline__ int find_sequence(const RowParams& P, uint32_t t, int lane, int& index) {
  if (!P.q_seqlens) {
    index = 0;
    return t < P.batch ? int(t) : -1;
  }
  const uint32_t tokens = uint32_t(P.tokens);  // < 2^31: two of them fit in 32 bits
  uint32_t before = 0;
  for (int b0 = 0; b0 < P.batch; b0 += 128) {
    uint32_t ends[4], sum = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int b = b0 + 4 * lane + j;
      const int n = b < P.batch ? max(P.q_seqlens[b], 0) : 0;
      ends[j] = sum = min(sum + min(uint32_t(n), tokens), tokens);
    }
    uint32_t upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t up = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto = min(upto + up, tokens);
    }
    // the first lane whose sequences end behind the token holds it
    const unsigned hit = __ballot_sync(0xffffffffu, t - before < upto);
    if (hit) {
      const int l = __ffs(hit) - 1;
      uint32_t start = __shfl_up_sync(0xffffffffu, upto, 1);
      if (lane == 0) start = 0;
      const uint32_t own = t - before - start;  // of lane l: below its `sum`
      int j = 0;
      uint32_t from = 0;
#pragma unroll
      for (int k = 0; k < 3; ++k)
        if (own >= ends[k]) j = k + 1, from = ends[k];
      index = int(__shfl_sync(0xffffffffu, own - from, l));
      return b0 + 4 * l + __shfl_sync(0xffffffffu, j, l);
    }
    before += __shfl_sync(0xffffffffu, upto, 31);  // at most t
  }
  return -1;
}

// What no token's warp can see of the lengths: that one is negative or past its bound, or
// that they are more than the tokens. One warp, launched where there is a status to tell and
// lengths to look at. (As a warp of the rows' own grid it took the ragged store from 47 to 51 us.)
__global__ void __launch_bounds__(32) lengths_kernel(const int32_t* q_seqlens, int batch, int max_rows,
                                                     uint32_t tokens, uint32_t* status) {
  const uint32_t over = tokens + 1;  // < 2^30: two of them fit in 32 bits
  uint32_t sum = 0;
  bool bad = false;
  for (int b = threadIdx.x; b < batch; b += 32) {
    const int q = q_seqlens ? q_seqlens[b] : 1;
    bad |= q < 0 || q > max_rows;
    sum = min(sum + min(uint32_t(max(q, 0)), over), over);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum = min(sum + __shfl_xor_sync(0xffffffffu, sum, o), over);
  if (bad || sum == over) report(status, PA_STATUS_BIT_PLAN);
}

// One warp per (token, slice of its query, key or value heads), U rows to a
// group of lanes. A row's elements are 16-byte chunks of 8; a lane holds chunk
// pair p: chunks p and p + rot / 16 where they are rotated (so that both members
// of every pair are its own, in either pairing), 2p and 2p + 1 behind the rotated
// part, and p and p + dims / 16 of a row that is not rotated at all. What a row
// is multiplied by but its own norm is the same for all rows of the warp: weight
// times cosine and weight times sine, made once.
//
// Bytes bound these rows, and come close: 8192 tokens of 32 + 8 heads of 128 are turned in
// 32.5 us (25.3 at the copy rate; issue slots 66 % full), and 2 x 32 heads of as many
// written to 8 bits in 37 (29.6; conversions and maxima keep the ALU 64 % busy). The store
// of 8 prompts of 1 to 2048 tokens, 48 heads, takes 47 us (51 with a cold cache) for 24 us of
// bytes: it makes the factors, looks the token up and quantises. Registers are held to what lets 32
// warps an SM (40 in the write) have loads in flight; a warp that loaded the next token's rows
// ahead, at half the warps, was slower (39 us for the 8192 tokens).
//
// AXES: the pairs' positions lie on several axes. Four pairs next to one another take their
// cosines in one load where they have one axis, as sections of at least eight pairs mostly do, else
// one by one.
template <int MODE, int VPL, int U, bool IL, bool AXES>
__global__ void __launch_bounds__(256, VPL == 1 ? (MODE == kWrite ? 5 : 4) : 1)
rows_kernel(const RowParams P) {
  const int lane = threadIdx.x & 31;
  const int lanes = 1 << P.lane_shift, per_warp = 32 >> P.lane_shift;
  const int group = lane >> P.lane_shift, gl = lane & (lanes - 1);
  const uint32_t task = blockIdx.x * 8u + (threadIdx.x >> 5);
  const int64_t t = task / P.slices;
  if (t >= P.tokens) return;
  const uint32_t slice = task - uint32_t(t) * P.slices;
  const bool is_q = MODE != kWrite && slice < P.q_slices;
  const bool is_v = MODE != kRotate && slice >= P.q_slices + P.k_slices;
  const bool turned = MODE != kWrite && !is_v;  // normed and rotated
  const int step = U * per_warp;  // rows of a batch
  const int first = int(slice - (is_q ? 0 : is_v ? P.q_slices + P.k_slices : P.q_slices)) * step * P.batches;
  int left = min((is_q ? P.heads : P.kv_heads) - first, step * P.batches);  // rows to do
  const int dims = is_v ? P.hv : P.hk;
  const int half = turned && P.rot ? P.rot / 16 : dims / 16;

  const __half* src = is_q   ? P.query + t * P.query_stride
                      : is_v ? P.value + t * P.value_stride
                             : P.key + t * P.key_stride;
  src += int64_t(first + group) * dims;
  int at[VPL][2];
  bool on[VPL], turn[VPL];
#pragma unroll
  for (int v = 0; v < VPL; ++v) {
    const int p = gl + v * lanes;
    on[v] = p < dims / 16;
    turn[v] = turned && p < P.rot / 16;
#pragma unroll
    for (int c = 0; c < 2; ++c) at[v][c] = p < half ? (p + c * half) * 8 : 16 * p + 8 * c;
  }

  // ---- a batch's elements: the first loads do not wait for where the token goes
  uint4 x[U][VPL][2];
  const auto load = [&] {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int v = 0; v < VPL; ++v)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          x[u][v][c] = make_uint4(0, 0, 0, 0);
          if (on[v] && u * per_warp + group < left)
            x[u][v][c] = *reinterpret_cast<const uint4*>(src + u * per_warp * dims + at[v][c]);
        }
    src += step * dims;
  };
  load();

  // ---- where the token goes
  int64_t slot = -1;
  int block = 0, place = 0, pos = 0;
  if constexpr (MODE == kRotate) {
    if (!AXES) pos = P.positions[t];
  } else {
    int i = 0;
    const int b = find_sequence(P, t, lane, i);
    if (b < 0) return;
    const int q = P.q_seqlens ? P.q_seqlens[b] : 1, L = P.context_lens[b];
    if (q > P.max_rows || L < q || int64_t(L) > int64_t(P.max_blocks_per_seq) * P.block_size) {
      if (L != 0 || P.q_seqlens) report(P.status, PA_STATUS_BIT_PLAN);  // (else padding)
      return;
    }
    pos = L - q + i;
    block = P.block_tables[int64_t(b) * P.max_blocks_per_seq + pos / P.block_size];
    place = pos % P.block_size;
    if (block >= 0 && block < P.num_blocks) slot = int64_t(block) * P.block_size + place;
    else report(P.status, PA_STATUS_BIT_BLOCK_INDEX);
    if (MODE == kStore && !AXES && P.positions) pos = P.positions[t];
  }
  int axis_pos[4];  // (AXES)
  if constexpr (AXES) {
    bool bad = false, out = false;
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      axis_pos[a] = a < P.axes ? P.positions[a * P.tokens + t] : 0;
      bad |= axis_pos[a] < -1 || axis_pos[a] >= P.max_positions;
      out |= axis_pos[a] < 0;
    }
    if (bad) report(P.status, PA_STATUS_BIT_POSITION);
    if (bad || out) return;
  } else if (MODE != kWrite) {
    if (pos < -1 || pos >= P.max_positions) report(P.status, PA_STATUS_BIT_POSITION);
    if (pos < 0 || pos >= P.max_positions) return;
  }

  // ---- the factors. Pair m of chunk pair v: elements m of both chunks, or
  // (interleaved) 2m and 2m + 1 of the 16; ca, cb: the cosine times the weight
  // of its first and second, sa, sb: the sine.
  // Keys on their way to 8 bits are rounded coarsely, and an error in the last place of fp32 that
  // moves one over a border costs a whole step; so they are made closer: an element times
  // its weight is exact in fp32 (11 bits times 11), the sum of two products is taken with the
  // error of one of them (Kahan), and ca, cb are the weights, sa, sb cosine and sine.
  const bool exact = MODE == kStore && !is_q;
  const auto chunk_of = [](int m, int second) { return IL ? m / 4 : second; };
  const auto elem_of = [](int m, int second) { return IL ? 2 * (m % 4) + second : m; };
  float ca[VPL][8], cb[VPL][8], sa[VPL][8], sb[VPL][8];
  const __half* weight = is_q ? P.q_weight : P.k_weight;
  if (turned) {
    const float* table = P.cos_sin + int64_t(pos) * P.rot;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      float w[2][8];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint4 g = make_uint4(0x3c003c00u, 0x3c003c00u, 0x3c003c00u, 0x3c003c00u);  // ones
        if (weight && on[v]) g = *reinterpret_cast<const uint4*>(weight + at[v][c]);
        const uint32_t* h = reinterpret_cast<const uint32_t*>(&g);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = h2f2(h[j]);
          w[c][2 * j] = f.x;
          w[c][2 * j + 1] = f.y;
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float4 cs = make_float4(1.f, 1.f, 1.f, 1.f), sn = make_float4(0.f, 0.f, 0.f, 0.f);
        if constexpr (AXES) {
          if (turn[v]) {
            const int i = IL ? at[v][c] / 2 : at[v][0] + 4 * c;  // the first of four pairs
            float* cw = reinterpret_cast<float*>(&cs);
            float* sw = reinterpret_cast<float*>(&sn);
            const uint32_t of = P.axis_of[i / 16] >> (i % 16 * 2) & 255;  // two bits each
            const float *cosines = P.cos_sin + i, *sines = cosines + P.rot / 2;
            const auto row = [&](uint32_t a) {  // where the position of axis a has its row
              return int64_t(a & 2 ? (a & 1 ? axis_pos[3] : axis_pos[2]) : (a & 1 ? axis_pos[1] : axis_pos[0])) * P.rot;
            };
            if (of == (of & 3) * 0x55) {
              cs = *reinterpret_cast<const float4*>(cosines + row(of));
              sn = *reinterpret_cast<const float4*>(sines + row(of));
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int64_t at = row(of >> 2 * j) + j;
                cw[j] = cosines[at];
                sw[j] = sines[at];
              }
            }
          }
        } else if (turn[v]) {
          const float* from = table + (IL ? at[v][c] / 2 : at[v][0] + 4 * c);
          cs = *reinterpret_cast<const float4*>(from);
          sn = *reinterpret_cast<const float4*>(from + P.rot / 2);
        }
        const float* cc = reinterpret_cast<const float*>(&cs);
        const float* ss = reinterpret_cast<const float*>(&sn);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int m = 4 * c + j;
          const float wa = w[chunk_of(m, 0)][elem_of(m, 0)], wb = w[chunk_of(m, 1)][elem_of(m, 1)];
          ca[v][m] = exact ? wa : wa * cc[j];
          cb[v][m] = exact ? wb : wb * cc[j];
          sa[v][m] = exact ? cc[j] : wa * ss[j];
          sb[v][m] = exact ? ss[j] : wb * ss[j];
        }
      }
    }
  }

  __half* dense = is_q            ? P.q_out + (t * P.heads + first + group) * P.hk
                  : MODE == kRotate ? P.k_out + (t * P.kv_heads + first + group) * P.hk
                                    : nullptr;
  const int64_t head0 = slot * P.kv_heads + first + group;
  uint8_t* codes = is_v ? P.value_cache + head0 * dims : P.key_cache + head0 * dims;
  uint8_t* exps = (is_v ? P.value_exps : P.key_exps) +
                  (int64_t(block) * P.kv_heads + first + group) * P.block_size + place;

#pragma unroll 1
  for (;;) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u * per_warp >= left) break;
      const bool row_on = u * per_warp + group < left;
      const int64_t row = u * per_warp;  // from the pointers on
      if (MODE != kWrite && turned) {
        float y[VPL][2][8], sq = 0.f, inv = 1.f;
#pragma unroll
        for (int v = 0; v < VPL; ++v)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(&x[u][v][c]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 f = h2f2(w[j]);
              y[v][c][2 * j] = f.x;
              y[v][c][2 * j + 1] = f.y;
              sq += f.x * f.x + f.y * f.y;
            }
          }
        if (weight) {
          #pragma unroll
          for (int o = 16; o; o >>= 1)
            if (o < lanes) sq += __shfl_xor_sync(0xffffffffu, sq, o);
          // one step of Newton's method takes rsqrtf's two units of error to one (a row with an
          // infinity has inv = 0, where the step's residual is NaN)
          const float mean = sq * P.inv_hk + P.eps;
          inv = rsqrtf(mean);
          const float rest = fmaf(-mean * inv, inv, 1.f);
          if (rest == rest) inv = fmaf(0.5f * inv, rest, inv);
        }
        if (exact) {
#pragma unroll
          for (int v = 0; v < VPL; ++v)
#pragma unroll
            for (int m = 0; m < 8; ++m) {
              float& fa = y[v][chunk_of(m, 0)][elem_of(m, 0)];
              float& fb = y[v][chunk_of(m, 1)][elem_of(m, 1)];
              const float a = fa * ca[v][m], b = fb * cb[v][m];
              fa = a;
              fb = b;
              if (turn[v]) {
                const float bs = b * sb[v][m], as = a * sb[v][m];
                fa = fmaf(a, sa[v][m], -bs) + fmaf(-b, sb[v][m], bs);
                fb = fmaf(b, sa[v][m], as) + fmaf(a, sb[v][m], -as);
              }
              fa *= inv;
              fb *= inv;
            }
        } else {
#pragma unroll
          for (int v = 0; v < VPL; ++v)
#pragma unroll
            for (int m = 0; m < 8; ++m) {
              float& fa = y[v][chunk_of(m, 0)][elem_of(m, 0)];
              float& fb = y[v][chunk_of(m, 1)][elem_of(m, 1)];
              const float a = fa * inv, b = fb * inv;
              // a sine of 0 is no reason to take in the other element's infinity
              fa = a * ca[v][m];
              fb = b * cb[v][m];
              if (turn[v]) {
                fa -= b * sb[v][m];
                fb += a * sa[v][m];
              }
            }
        }
        if (MODE == kRotate || is_q) {  // fp16 rows
#pragma unroll
          for (int v = 0; v < VPL; ++v)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float* f = y[v][c];
              if (on[v] && row_on)
                *reinterpret_cast<uint4*>(dense + row * dims + at[v][c]) =
                    make_uint4(pack_half2(f[0], f[1]), pack_half2(f[2], f[3]),
                               pack_half2(f[4], f[5]), pack_half2(f[6], f[7]));
            }
          continue;
        }
        // 8-bit rows: the exponent that the row's largest finite element needs,
        // then the codes (scaling by a power of two is exact). fmaxf leaves NaN
        // out; an infinity, which is rare, is made one and left out so.
        const auto largest = [&] {
          float top = 0.f;
#pragma unroll
          for (int v = 0; v < VPL; ++v)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(y[v][c][j]));
          for (int o = lanes >> 1; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          return top;
        };
        float top = largest();
        if (__any_sync(0xffffffffu, isinf(top))) {
#pragma unroll
          for (int v = 0; v < VPL; ++v)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (isinf(y[v][c][j])) y[v][c][j] = __uint_as_float(0x7fc00000u);
          top = largest();
        }
        const int e = row_exponent(top);
        const float f = pow2(-e);
#pragma unroll
        for (int v = 0; v < VPL; ++v)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float* a = y[v][c];
            const uint32_t lo = e4m3x2(a[0] * f, a[1] * f) | e4m3x2(a[2] * f, a[3] * f) << 16;
            const uint32_t hi = e4m3x2(a[4] * f, a[5] * f) | e4m3x2(a[6] * f, a[7] * f) << 16;
            if (on[v] && row_on && slot >= 0)
              *reinterpret_cast<uint2*>(codes + row * dims + at[v][c]) = make_uint2(lo, hi);
          }
        if (gl == 0 && row_on && slot >= 0) exps[row * P.block_size] = uint8_t(e + kExpBias);
      } else if (MODE != kRotate) {
        // Rows that are only quantised stay fp16, two elements to an
        // instruction. Times 2^-e an element is exact or ends below 2^-14, and
        // the least code is 2^-9: both give 0.
        uint32_t y[VPL][2][4];
#pragma unroll
        for (int v = 0; v < VPL; ++v)
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) y[v][c][j] = reinterpret_cast<const uint32_t*>(&x[u][v][c])[j];
        const auto largest = [&] {
          uint32_t top = 0;
#pragma unroll
          for (int v = 0; v < VPL; ++v)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int j = 0; j < 4; ++j) top = max_half2(top, y[v][c][j] & 0x7fff7fffu);
          for (int o = lanes >> 1; o; o >>= 1)
            top = max_half2(top, __shfl_xor_sync(0xffffffffu, top, o));
          const float2 f = h2f2(top);
          return fmaxf(f.x, f.y);
        };
        float top = largest();
        if (__any_sync(0xffffffffu, isinf(top))) {
#pragma unroll
          for (int v = 0; v < VPL; ++v)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t& w = y[v][c][j];
                if ((w & 0x7fffu) == 0x7c00u) w |= 0x200u;
                if ((w >> 16 & 0x7fffu) == 0x7c00u) w |= 0x2000000u;
              }
          top = largest();
        }
        const int e = row_exponent(top);  // in [-32, 8]; fp16 has the powers up to 15
#pragma unroll 1
        for (int more = -e; ; more -= 15) {
          const uint32_t f = half2_pow2(min(max(more, -14), 15));
#pragma unroll
          for (int v = 0; v < VPL; ++v)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int j = 0; j < 4; ++j) y[v][c][j] = mul_half2(y[v][c][j], f);
          if (!__any_sync(0xffffffffu, more > 15)) break;
          if (more < 15) more = 15;  // this row is done: 2^0 from here on
        }
#pragma unroll
        for (int v = 0; v < VPL; ++v)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t* a = y[v][c];
            const uint32_t lo = half2_e4m3x2(a[0]) | half2_e4m3x2(a[1]) << 16;
            const uint32_t hi = half2_e4m3x2(a[2]) | half2_e4m3x2(a[3]) << 16;
            if (on[v] && row_on && slot >= 0)
              *reinterpret_cast<uint2*>(codes + row * dims + at[v][c]) = make_uint2(lo, hi);
          }
        if (gl == 0 && row_on && slot >= 0) exps[row * P.block_size] = uint8_t(e + kExpBias);
      }
    }
    if ((left -= step) <= 0) return;
    load();
    dense += int64_t(step) * dims;
    codes += int64_t(step) * dims;
    exps += int64_t(step) * P.block_size;
  }
}

template <int MODE, bool IL, bool AXES = false>
pa_status launch_rows(RowParams P, cudaStream_t stream) {
  if (P.tokens == 0) return PA_OK;
  if (P.tokens > INT32_MAX) return PA_ERR_INVALID_ARG;  // (before it is multiplied)
  const int widest = (MODE == kRotate || P.hk > P.hv ? P.hk : P.hv) / 16;  // chunk pairs of a row
  while ((1 << P.lane_shift) < widest && P.lane_shift < 5) ++P.lane_shift;
  P.inv_hk = 1.0f / float(P.hk);
  const int per_warp = 32 >> P.lane_shift;
  const auto slice = [&](int rows) {
    P.q_slices = MODE == kWrite ? 0 : uint32_t(cdiv(P.heads, rows));
    P.k_slices = uint32_t(cdiv(P.kv_heads, rows));
    P.slices = P.q_slices + P.k_slices * (MODE == kRotate ? 1 : 2);
    return P.tokens * P.slices;
  };
  const bool many = widest <= 32 && slice(per_warp * kRows * kBatches) >= kManyWarps;
  P.batches = many ? kBatches : 1;
  if (!many) slice(per_warp);
  if (P.tokens * P.slices > INT32_MAX) return PA_ERR_INVALID_ARG;
  const unsigned grid = unsigned(cdiv(P.tokens * P.slices, 8));
  if (many) rows_kernel<MODE, 1, kRows, IL, AXES><<<grid, 256, 0, stream>>>(P);
  else if (widest <= 32) rows_kernel<MODE, 1, 1, IL, AXES><<<grid, 256, 0, stream>>>(P);
  else rows_kernel<MODE, 2, 1, IL, AXES><<<grid, 256, 0, stream>>>(P);
  if (MODE != kRotate && P.status && (P.q_seqlens || P.batch > P.tokens))
    lengths_kernel<<<1, 32, 0, stream>>>(P.q_seqlens, P.batch, P.max_rows, uint32_t(P.tokens), P.status);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

template <int MODE>
pa_status launch_turned(const RowParams& P, cudaStream_t s) {
  if (P.axes) return P.interleaved ? launch_rows<MODE, true, true>(P, s) : launch_rows<MODE, false, true>(P, s);
  return P.interleaved ? launch_rows<MODE, true>(P, s) : launch_rows<MODE, false>(P, s);
}

// ---- reading back

struct ReadParams {
  const uint8_t *key_cache, *key_exps, *value_cache, *value_exps;
  const int32_t *block_tables, *starts, *context_lens, *out_starts;
  __half *k_out, *v_out;
  uint32_t* status;
  int64_t out_rows;
  int batch, kv_heads, hk, hv, block_size, num_blocks, max_blocks_per_seq, max_rows;
  int k_slices, v_slices;  // warps of a token's keys and of its values
  int strip;               // tokens of a warp, at most 32
};

// Eight codes times 2^(byte - 127), rounded once to fp16. Within [-14, 15] the
// power is an fp16 and one product rounds once. Elsewhere the power is split:
// the first product is exact (a code is a multiple of 2^-9, so that times 2^-14
// it is one of 2^-23) or infinite as the result is, and the second rounds. Powers
// past [-38, 30] give the zeros and infinities that these ends give.
__device__ __forceinline__ uint4 widen(const uint2& codes, int byte) {
  const int e = byte - kExpBias, near = min(max(e, -14), 15);
  const uint32_t f = half2_pow2(near);
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    o[j] = mul_half2(e4m3x2_half2((j < 2 ? codes.x : codes.y) >> (j % 2 ? 16 : 0)), f);
  if (e != near) {
    const __half2 g = __float2half2_rn(pow2(min(max(e - near, -24), 15)));
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = mul_half2(o[j], *reinterpret_cast<const uint32_t*>(&g));
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// One warp per (strip of tokens of a sequence, 1 KB of their keys or of
// their values): a token's heads are contiguous in the cache and in the output.
// Lane l finds token l's place, so that a strip waits for one table lookup. A
// lane reads 8 codes and writes 16 bytes, neighbouring lanes neighbouring ones.
// 32 sequences of 64 to 8192 tokens, 8 + 8 heads of 128, come back in 146 us, 6.1 TB/s of
// reads and writes (90 % of a copy), with a token at a time and 40 warps an SM; with
// four tokens at a time and 16 warps it took 190.
__global__ void __launch_bounds__(256, 5) read_kernel(const ReadParams P) {
  constexpr int kUnroll = 4;
  const int lane = threadIdx.x & 31;
  const int slices = P.k_slices + P.v_slices;
  for (int b = blockIdx.y; b < P.batch; b += gridDim.y) {
    const int start = P.starts ? P.starts[b] : 0, L = P.context_lens[b];
    if (start < 0 || L < start || int64_t(L) > int64_t(P.max_blocks_per_seq) * P.block_size ||
        L - start > P.max_rows) {
      if (threadIdx.x == 0) report(P.status, PA_STATUS_BIT_PLAN);
      continue;
    }
    const int64_t out0 = P.out_starts[b], tasks = (int64_t(L - start) + P.strip - 1) / P.strip * slices;
    for (int64_t k = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); k < tasks; k += int64_t(gridDim.x) * 8) {
      const int64_t strip = k <= UINT32_MAX ? uint32_t(k) / uint32_t(slices) : k / slices;
      const int slice = int(k - strip * slices), i0 = int(strip) * P.strip;
      const int rows = min(P.strip, L - start - i0);
      const bool kv = slice >= P.k_slices;
      const int hd = kv ? P.hv : P.hk, width = P.kv_heads * hd, n = hd / 8;
      const int c0 = (kv ? slice - P.k_slices : slice) * (32 * kUnroll) + lane;
      const int chunks = (width / 8 - c0 + 31) / 32;  // of this lane in a row, from c0 on
      const uint8_t* cache = (kv ? P.value_cache : P.key_cache) + c0 * 8;
      __half* dst = (kv ? P.v_out : P.k_out) + (out0 + i0) * width + c0 * 8;

      // token `lane` of the strip: its slot, and where its exponents begin
      int slot = -1;
      int64_t first = 0;
      if (lane < rows) {
        const int pos = start + i0 + lane;
        const int64_t out = out0 + i0 + lane;
        if (out < 0 || out >= P.out_rows) {
          report(P.status, PA_STATUS_BIT_WORKSPACE);
        } else {
          const int page = pos / P.block_size, place = pos - page * P.block_size;
          const int block = P.block_tables[int64_t(b) * P.max_blocks_per_seq + page];
          if (block >= 0 && block < P.num_blocks) {
            slot = block * P.block_size + place;
            first = int64_t(block) * P.kv_heads * P.block_size + place;
          } else {
            report(P.status, PA_STATUS_BIT_BLOCK_INDEX);
          }
        }
      }
      const uint8_t* exps[kUnroll];  // of the heads of this lane's chunks
      int h = c0 / n, rest = c0 - h * n;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        exps[u] = (kv ? P.value_exps : P.key_exps) + int64_t(h) * P.block_size;
        rest += 32 % n;
        h += 32 / n;
        if (rest >= n) rest -= n, ++h;
      }

      for (int r = 0; r < rows; ++r, dst += width) {
        const int64_t at = __shfl_sync(0xffffffffu, slot, r);
        const int64_t f = __shfl_sync(0xffffffffu, first, r);
        if (at < 0) continue;
        uint2 codes[kUnroll];
        int e[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (u < chunks) {
            codes[u] = *reinterpret_cast<const uint2*>(cache + at * width + 256 * u);
            e[u] = exps[u][f];
          }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (u < chunks) *reinterpret_cast<uint4*>(dst + 256 * u) = widen(codes[u], e[u]);
      }
    }
  }
}

// ---- host checks

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

bool head_size_ok(int hs) { return hs > 0 && hs <= PA_MAX_HEAD_SIZE && hs % 16 == 0; }

pa_status check_cache(const pa_cache_config* c, const void* k, const void* ke, const void* v,
                      const void* ve, const int32_t* tables, const int32_t* lens) {
  if (!c || !k || !ke || !v || !ve || !tables || !lens) return PA_ERR_INVALID_ARG;
  if (c->batch <= 0 || c->batch > PA_MAX_BATCH || c->kv_heads <= 0) return PA_ERR_INVALID_ARG;
  if (!head_size_ok(c->head_size_k) || !head_size_ok(c->head_size_v)) return PA_ERR_INVALID_ARG;
  if (c->block_size <= 0 || c->block_size % 16 || c->num_blocks <= 0 || c->max_blocks_per_seq <= 0 ||
      c->max_rows < 0)
    return PA_ERR_INVALID_ARG;
  if (int64_t(c->num_blocks) * c->block_size > INT32_MAX) return PA_ERR_INVALID_ARG;
  if (int64_t(c->kv_heads) * PA_MAX_HEAD_SIZE > INT32_MAX) return PA_ERR_INVALID_ARG;
  if (k == v || ke == ve) return PA_ERR_INVALID_ARG;  // two caches, each with its own exponents
  if (!aligned16(k) || !aligned16(ke) || !aligned16(v) || !aligned16(ve)) return PA_ERR_INVALID_ARG;
  return PA_OK;
}

pa_status check_rotary(const pa_rotary* r, const void* q_weight, const void* k_weight,
                       const float* cos_sin) {
  if (!r || r->num_heads <= 0 || r->kv_heads <= 0 || !head_size_ok(r->head_size))
    return PA_ERR_INVALID_ARG;
  if (int64_t(r->num_heads) + 2 * int64_t(r->kv_heads) > INT32_MAX / PA_MAX_HEAD_SIZE)
    return PA_ERR_INVALID_ARG;
  if (r->rotary_dim < 0 || r->rotary_dim > r->head_size || r->rotary_dim % 16 ||
      r->max_positions <= 0)
    return PA_ERR_INVALID_ARG;
  if (!(r->eps >= 0.f) || std::isinf(r->eps)) return PA_ERR_INVALID_ARG;
  if (r->rotary_dim > 0 && !cos_sin) return PA_ERR_INVALID_ARG;
  if (!aligned16(q_weight) || !aligned16(k_weight) || !aligned16(cos_sin)) return PA_ERR_INVALID_ARG;
  return PA_OK;
}

pa_status check_axes(const pa_axes* a, const pa_rotary* r, const int32_t* positions) {
  if (!a || !positions || a->count < 1 || a->count > PA_MAX_AXES) return PA_ERR_INVALID_ARG;
  const int64_t pairs = r->rotary_dim / 2;
  int64_t sum = 0;
  for (int i = 0; i < a->count; ++i) {
    const int64_t n = a->sections[i];
    if (n < 0 || (a->cyclic && i && n && a->count * (n - 1) + i >= pairs)) return PA_ERR_INVALID_ARG;
    sum += n;
  }
  return sum == pairs ? PA_OK : PA_ERR_INVALID_ARG;
}

void set_axes(RowParams& P, const pa_axes& a) {
  P.axes = a.count;
  int axis = 0, left = a.sections[0];  // of the sections behind one another
  for (int i = 0; i < P.rot / 2; ++i) {
    if (a.cyclic) {
      axis = i % a.count;
      if (i >= a.count * int64_t(a.sections[axis])) axis = 0;
    } else {
      while (left == 0) left = a.sections[++axis];
      --left;
    }
    P.axis_of[i / 16] |= uint32_t(axis) << (i % 16 * 2);
  }
}

// A row tensor: head h of token t at [t * stride + h * hs].
pa_status check_rows(const void* p, int64_t stride, int64_t width) {
  if (!p || !aligned16(p) || stride % 8 || stride < width) return PA_ERR_INVALID_ARG;
  return PA_OK;
}

void set_rotary(RowParams& P, const pa_rotary& r, const void* q_weight, const void* k_weight,
                const float* cos_sin, const int32_t* positions) {
  P.heads = r.num_heads;
  P.kv_heads = r.kv_heads;
  P.hk = r.head_size;
  P.rot = r.rotary_dim;
  P.interleaved = r.interleaved;
  P.max_positions = r.max_positions;
  P.eps = r.eps;
  P.q_weight = static_cast<const __half*>(q_weight);
  P.k_weight = static_cast<const __half*>(k_weight);
  P.cos_sin = cos_sin;
  P.positions = positions;
}

void set_cache(RowParams& P, const pa_cache_config& c, const int32_t* block_tables,
               const int32_t* context_lens, const int32_t* q_seqlens, void* key_cache,
               uint8_t* key_exps, void* value_cache, uint8_t* value_exps) {
  P.batch = c.batch;
  P.kv_heads = c.kv_heads;
  P.hk = c.head_size_k;
  P.hv = c.head_size_v;
  P.block_size = c.block_size;
  P.num_blocks = c.num_blocks;
  P.max_blocks_per_seq = c.max_blocks_per_seq;
  P.max_rows = q_seqlens ? c.max_rows : 1;
  P.block_tables = block_tables;
  P.context_lens = context_lens;
  P.q_seqlens = q_seqlens;
  P.key_cache = static_cast<uint8_t*>(key_cache);
  P.key_exps = key_exps;
  P.value_cache = static_cast<uint8_t*>(value_cache);
  P.value_exps = value_exps;
}

}  // namespace

}  // namespace pa

namespace pa {

namespace {

// pa_qk_norm_rope, and pa_qk_norm_rope_axes with `axes`.
pa_status norm_rope(const pa_rotary* rot, const pa_axes* axes, bool with_axes, int64_t tokens, const void* query,
                    int64_t query_stride, const void* key, int64_t key_stride, const void* q_weight,
                    const void* k_weight, const float* cos_sin, const int32_t* positions, void* q_out, void* k_out,
                    uint32_t* status, void* stream) {
  pa_status st = check_rotary(rot, q_weight, k_weight, cos_sin);
  if (st == PA_OK && with_axes) st = check_axes(axes, rot, positions);
  if (st != PA_OK) return st;
  const int64_t qw = int64_t(rot->num_heads) * rot->head_size;
  const int64_t kw = int64_t(rot->kv_heads) * rot->head_size;
  if (tokens < 0 || !positions || !q_out || !k_out || !aligned16(q_out) || !aligned16(k_out))
    return PA_ERR_INVALID_ARG;
  if ((st = check_rows(query, query_stride, qw)) != PA_OK) return st;
  if ((st = check_rows(key, key_stride, kw)) != PA_OK) return st;
  if ((q_out == query && query_stride != qw) || (k_out == key && key_stride != kw) || q_out == k_out)
    return PA_ERR_INVALID_ARG;
  RowParams P{};
  set_rotary(P, *rot, q_weight, k_weight, cos_sin, positions);
  P.tokens = tokens;
  P.query = static_cast<const __half*>(query);
  P.key = static_cast<const __half*>(key);
  P.query_stride = query_stride;
  P.key_stride = key_stride;
  P.q_out = static_cast<__half*>(q_out);
  P.k_out = static_cast<__half*>(k_out);
  P.status = status;
  if (with_axes) set_axes(P, *axes);
  return launch_turned<kRotate>(P, static_cast<cudaStream_t>(stream));
}

// pa_cache_store, and pa_cache_store_axes with `axes`.
pa_status store(const pa_cache_config* cfg, const pa_rotary* rot, const pa_axes* axes, bool with_axes, int64_t tokens,
                const void* query, int64_t query_stride, const void* key, int64_t key_stride, const void* value,
                int64_t value_stride, const void* q_weight, const void* k_weight, const float* cos_sin,
                const int32_t* positions, const int32_t* block_tables, const int32_t* context_lens,
                const int32_t* q_seqlens, void* key_cache, uint8_t* key_exps, void* value_cache, uint8_t* value_exps,
                void* q_out, uint32_t* status, void* stream) {
  pa_status st = check_cache(cfg, key_cache, key_exps, value_cache, value_exps, block_tables, context_lens);
  if (st != PA_OK) return st;
  if ((st = check_rotary(rot, q_weight, k_weight, cos_sin)) != PA_OK) return st;
  if (with_axes && (st = check_axes(axes, rot, positions)) != PA_OK) return st;
  if (rot->kv_heads != cfg->kv_heads || rot->head_size != cfg->head_size_k) return PA_ERR_INVALID_ARG;
  const int64_t qw = int64_t(rot->num_heads) * rot->head_size;
  if (tokens < 0 || !q_out || !aligned16(q_out) || (q_out == query && query_stride != qw))
    return PA_ERR_INVALID_ARG;
  if ((st = check_rows(query, query_stride, qw)) != PA_OK) return st;
  if ((st = check_rows(key, key_stride, int64_t(cfg->kv_heads) * cfg->head_size_k)) != PA_OK) return st;
  if ((st = check_rows(value, value_stride, int64_t(cfg->kv_heads) * cfg->head_size_v)) != PA_OK) return st;
  RowParams P{};
  set_rotary(P, *rot, q_weight, k_weight, cos_sin, positions);
  set_cache(P, *cfg, block_tables, context_lens, q_seqlens, key_cache, key_exps, value_cache, value_exps);
  P.tokens = tokens;
  P.query = static_cast<const __half*>(query);
  P.key = static_cast<const __half*>(key);
  P.value = static_cast<const __half*>(value);
  P.query_stride = query_stride;
  P.key_stride = key_stride;
  P.value_stride = value_stride;
  P.q_out = static_cast<__half*>(q_out);
  P.status = status;
  if (with_axes) set_axes(P, *axes);
  return launch_turned<kStore>(P, static_cast<cudaStream_t>(stream));
}

}  // namespace

}  // namespace pa

extern "C" pa_status pa_qk_norm_rope(const pa_rotary* rot, int64_t tokens, const void* query,
                                     int64_t query_stride, const void* key, int64_t key_stride,
                                     const void* q_weight, const void* k_weight,
                                     const float* cos_sin, const int32_t* positions, void* q_out,
                                     void* k_out, uint32_t* status, void* stream) {
  return pa::norm_rope(rot, nullptr, false, tokens, query, query_stride, key, key_stride, q_weight, k_weight, cos_sin,
                       positions, q_out, k_out, status, stream);
}

extern "C" pa_status pa_qk_norm_rope_axes(const pa_rotary* rot, const pa_axes* axes, int64_t tokens, const void* query,
                                          int64_t query_stride, const void* key, int64_t key_stride,
                                          const void* q_weight, const void* k_weight, const float* cos_sin,
                                          const int32_t* positions, void* q_out, void* k_out, uint32_t* status,
                                          void* stream) {
  return pa::norm_rope(rot, axes, true, tokens, query, query_stride, key, key_stride, q_weight, k_weight, cos_sin,
                       positions, q_out, k_out, status, stream);
}

extern "C" pa_status pa_cache_write(const pa_cache_config* cfg, int64_t tokens, const void* key,
                                    int64_t key_stride, const void* value, int64_t value_stride,
                                    const int32_t* block_tables, const int32_t* context_lens,
                                    const int32_t* q_seqlens, void* key_cache, uint8_t* key_exps,
                                    void* value_cache, uint8_t* value_exps, uint32_t* status,
                                    void* stream) {
  using namespace pa;
  pa_status st = check_cache(cfg, key_cache, key_exps, value_cache, value_exps, block_tables, context_lens);
  if (st != PA_OK) return st;
  if (tokens < 0) return PA_ERR_INVALID_ARG;
  if ((st = check_rows(key, key_stride, int64_t(cfg->kv_heads) * cfg->head_size_k)) != PA_OK) return st;
  if ((st = check_rows(value, value_stride, int64_t(cfg->kv_heads) * cfg->head_size_v)) != PA_OK) return st;
  RowParams P{};
  set_cache(P, *cfg, block_tables, context_lens, q_seqlens, key_cache, key_exps, value_cache, value_exps);
  P.tokens = tokens;
  P.key = static_cast<const __half*>(key);
  P.value = static_cast<const __half*>(value);
  P.key_stride = key_stride;
  P.value_stride = value_stride;
  P.status = status;
  return launch_rows<kWrite, false>(P, static_cast<cudaStream_t>(stream));
}

extern "C" pa_status pa_cache_store(const pa_cache_config* cfg, const pa_rotary* rot, int64_t tokens,
                                    const void* query, int64_t query_stride, const void* key,
                                    int64_t key_stride, const void* value, int64_t value_stride,
                                    const void* q_weight, const void* k_weight,
                                    const float* cos_sin, const int32_t* positions,
                                    const int32_t* block_tables, const int32_t* context_lens,
                                    const int32_t* q_seqlens, void* key_cache, uint8_t* key_exps,
                                    void* value_cache, uint8_t* value_exps, void* q_out,
                                    uint32_t* status, void* stream) {
  return pa::store(cfg, rot, nullptr, false, tokens, query, query_stride, key, key_stride, value, value_stride, q_weight,
                   k_weight, cos_sin, positions, block_tables, context_lens, q_seqlens, key_cache, key_exps,
                   value_cache, value_exps, q_out, status, stream);
}

extern "C" pa_status pa_cache_store_axes(const pa_cache_config* cfg, const pa_rotary* rot, const pa_axes* axes,
                                         int64_t tokens, const void* query, int64_t query_stride, const void* key,
                                         int64_t key_stride, const void* value, int64_t value_stride,
                                         const void* q_weight, const void* k_weight, const float* cos_sin,
                                         const int32_t* positions, const int32_t* block_tables,
                                         const int32_t* context_lens, const int32_t* q_seqlens, void* key_cache,
                                         uint8_t* key_exps, void* value_cache, uint8_t* value_exps, void* q_out,
                                         uint32_t* status, void* stream) {
  return pa::store(cfg, rot, axes, true, tokens, query, query_stride, key, key_stride, value, value_stride, q_weight,
                   k_weight, cos_sin, positions, block_tables, context_lens, q_seqlens, key_cache, key_exps,
                   value_cache, value_exps, q_out, status, stream);
}

extern "C" pa_status pa_cache_read(const pa_cache_config* cfg, const void* key_cache,
                                   const uint8_t* key_exps, const void* value_cache,
                                   const uint8_t* value_exps, const int32_t* block_tables,
                                   const int32_t* starts, const int32_t* context_lens,
                                   const int32_t* out_starts, int64_t out_rows, void* k_out,
                                   void* v_out, uint32_t* status, void* stream) {
  using namespace pa;
  const pa_status st =
      check_cache(cfg, key_cache, key_exps, value_cache, value_exps, block_tables, context_lens);
  if (st != PA_OK) return st;
  if (!out_starts || out_rows < 0 || !k_out || !v_out || k_out == v_out || !aligned16(k_out) ||
      !aligned16(v_out))
    return PA_ERR_INVALID_ARG;
  if (cfg->max_rows == 0 || out_rows == 0) return PA_OK;
  ReadParams P{};
  P.key_cache = static_cast<const uint8_t*>(key_cache);
  P.key_exps = key_exps;
  P.value_cache = static_cast<const uint8_t*>(value_cache);
  P.value_exps = value_exps;
  P.block_tables = block_tables;
  P.starts = starts;
  P.context_lens = context_lens;
  P.out_starts = out_starts;
  P.k_out = static_cast<__half*>(k_out);
  P.v_out = static_cast<__half*>(v_out);
  P.status = status;
  P.out_rows = out_rows;
  P.batch = cfg->batch;
  P.kv_heads = cfg->kv_heads;
  P.hk = cfg->head_size_k;
  P.hv = cfg->head_size_v;
  P.block_size = cfg->block_size;
  P.num_blocks = cfg->num_blocks;
  P.max_blocks_per_seq = cfg->max_blocks_per_seq;
  P.max_rows = cfg->max_rows;
  P.k_slices = int(cdiv(int64_t(cfg->kv_heads) * cfg->head_size_k, 1024));
  P.v_slices = int(cdiv(int64_t(cfg->kv_heads) * cfg->head_size_v, 1024));
  const int64_t slices = int64_t(P.k_slices) + P.v_slices;
  // a strip of tokens to a warp where that leaves warps enough
  P.strip = 16;
  while (P.strip > 1 && cdiv(cfg->max_rows, P.strip) * slices * cfg->batch < kManyWarps) P.strip /= 2;
  const int64_t tasks = cdiv(cfg->max_rows, P.strip) * slices;
  const dim3 grid(unsigned(std::min<int64_t>(cdiv(tasks, 8), 65536)),
                  unsigned(std::min(cfg->batch, 65535)));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  read_kernel<<<grid, 256, 0, s>>>(P);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
