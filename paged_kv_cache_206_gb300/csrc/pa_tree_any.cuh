// The attention kernel of pa_tree_forward and pa_window_forward for the largest heads.
#pragma once

#include "pa_tree.cuh"

namespace pa {

constexpr int kAnyWarps = 4;
constexpr int kAnyChunks = (PA_MAX_HEAD_SIZE / 8 + 31) / 32;  // 8-dim chunks a lane may hold
constexpr int kAnyFold = 64;  // keys that a warp sums before it adds them to its others
// A row's reference moves when a score passes it by 2^8 (base-2 exponents): what a move rounds away of the sums
// before it, they have shrunk by that much.
constexpr float kAnyMove = 8.f;

// Adds x to the sum s, what that rounds away to `lost` (Knuth's two-sum: exact as long as nothing overflows).
__device__ __forceinline__ void add_two_sum(float& s, float& lost, float x) {
  const float t = s + x, y = t - s;
  lost += (s - (t - y)) + (x - y);
  s = t;
}

// 8 elements of a cache row as they are held, and as fp32.
template <bool Q8>
__device__ __forceinline__ uint4 fetch8(const uint8_t* row, int d) {
  if constexpr (Q8) {
    const uint2 c = *reinterpret_cast<const uint2*>(row + d);
    return make_uint4(c.x, c.y, 0, 0);
  } else {
    return *reinterpret_cast<const uint4*>(row + 2 * d);
  }
}
template <bool Q8>
__device__ __forceinline__ void widen8(uint4 c, float (&x)[8]) {
  uint32_t h[4] = {c.x, c.y, c.z, c.w};
  if constexpr (Q8) {
    h[0] = e4m3x2_half2(c.x);
    h[1] = e4m3x2_half2(c.x >> 16);
    h[2] = e4m3x2_half2(c.y);
    h[3] = e4m3x2_half2(c.y >> 16);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = h2f2(h[j]);
    x[2 * j] = f.x;
    x[2 * j + 1] = f.y;
  }
}

// The lengths of sequences that no token of the call may belong to (one warp).
inline __device__ __noinline__ void tree_check_lengths(const TreeParams& P, int lane) {
  int64_t sum = 0;
  for (int b = lane; b < P.batch; b += 32) {
    const int q = P.q_seqlens ? P.q_seqlens[b] : 1;
    const int L = P.context_lens[b];
    if (!tree_lengths_ok(P, q, L) && !tree_padding(P, L)) set_status(P.status, PA_STATUS_BIT_PLAN);
    sum += max(q, 0);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (sum > P.tokens) set_status(P.status, PA_STATUS_BIT_PLAN);
}

// Heads of more than 256 dims. One CTA per (token, head); warp w takes the keys w, w + 4,
// ..., a lane holds 8-dim chunks lane, lane + 32, ... of the row. Softmax and sums in fp32.
// Bound by the latency of a key after another, and the heads of a group read the
// same keys each: 2.57 ms for 64 decode steps of up to 4096 keys, 32 heads of 272 dims on 8, 2.52 over
// 8 bits (3.3 and 3.4 with a key's value fetched behind its score). WIN: the keys are the sinks before the window,
// then those of the window.
//
// A warp adds up kAnyFold keys at a time and these sums to those of all its keys with what the additions
// round away kept beside: the error does not grow with the keys. (One by one, equal values over 2^20 keys came out
// 0.4 % off.)
template <bool Q8, bool WIN>
__global__ void __launch_bounds__(kAnyWarps * 32, 5) tree_any_kernel(const TreeParams P) {
  __shared__ float o_s[kAnyWarps][PA_MAX_HEAD_SIZE], lost_s[kAnyWarps][PA_MAX_HEAD_SIZE];
  __shared__ float m_s[kAnyWarps], l_s[kAnyWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x / P.num_heads;
  const int h = int(blockIdx.x % P.num_heads), kvh = h / P.group;
  int i;
  if (blockIdx.x == 0 && warp == 0) tree_check_lengths(P, lane);
  const int b = tree_sequence(P, t, lane, i);
  if (b < 0) return;
  const int q = P.q_seqlens ? P.q_seqlens[b] : 1, L = P.context_lens[b];
  if (!tree_lengths_ok(P, q, L)) {
    if (!tree_padding(P, L)) set_status(P.status, PA_STATUS_BIT_PLAN);
    return;
  }
  const int prefix = L - q;
  uint32_t bits[kTreeWords];
  if (!WIN && P.parents) tree_ancestors(P, P.parents + (t - i), i, bits);

  // pl, po: sums over the last kAnyFold keys, of weights 2^(score - m); l, o_s: over the keys before them, of
  // weights 2^(score - m_folded)
  float query[kAnyChunks][8], po[kAnyChunks][8];
#pragma unroll
  for (int k = 0; k < kAnyChunks; ++k) {
    const int d = (lane + 32 * k) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) query[k][j] = 0.f;
    if (d < P.hk)
      widen8<false>(fetch8<false>(reinterpret_cast<const uint8_t*>(P.query + (t * P.num_heads + h) * P.hk), d), query[k]);
    if (d < P.hv)
#pragma unroll
      for (int j = 0; j < 8; ++j) o_s[warp][d + j] = lost_s[warp][d + j] = 0.f;
  }
  float m = -INFINITY, m_folded = -INFINITY, l = 0.f, l_lost = 0.f;
  const int lo = WIN ? max(prefix + i - P.window + 1, 0) : 0, far = WIN ? min(P.sinks, lo) : 0;
  const int keys = prefix + i + 1 - (lo - far);
  for (int n0 = warp; n0 < keys; n0 += kAnyWarps * kAnyFold) {
    float pl = 0.f;
#pragma unroll
    for (int k = 0; k < kAnyChunks; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) po[k][e] = 0.f;
    for (int n = n0; n < min(n0 + kAnyWarps * kAnyFold, keys); n += kAnyWarps) {
      const int j = n < far ? n : n + (lo - far);
      if (!WIN && P.parents && j >= prefix) {
        const int a = j - prefix;
        if (!(bits[a >> 5] >> (a & 31) & 1)) continue;
      }
      const int block = P.block_tables[int64_t(b) * P.max_blocks_per_seq + j / P.block_size];
      if (block < 0 || block >= P.num_blocks) {
        if (lane == 0) set_status(P.status, PA_STATUS_BIT_BLOCK_INDEX);
        continue;
      }
      const int place = j % P.block_size;
      const int64_t row = (int64_t(block) * P.block_size + place) * P.kv_heads + kvh;
      const uint8_t* kr = P.key_cache + row * P.hk * (Q8 ? 1 : 2);
      const uint8_t* vr = P.value_cache + row * P.hv * (Q8 ? 1 : 2);
      uint4 value[kAnyChunks];  // on its way while the score is made
#pragma unroll
      for (int k = 0; k < kAnyChunks; ++k) {
        const int d = (lane + 32 * k) * 8;
        if (d < P.hv) value[k] = fetch8<Q8>(vr, d);
      }
      float dot = 0.f;
#pragma unroll
      for (int k = 0; k < kAnyChunks; ++k) {
        const int d = (lane + 32 * k) * 8;
        if (d >= P.hk) break;
        float x[8];
        widen8<Q8>(fetch8<Q8>(kr, d), x);
#pragma unroll
        for (int e = 0; e < 8; ++e) dot += query[k][e] * x[e];
      }
      float s = warp_sum(dot) * P.scale_log2;
      float vscale = 1.f;
      if constexpr (Q8) {
        const int64_t at = (int64_t(block) * P.kv_heads + kvh) * P.block_size + place;
        s *= pow2(int(P.key_exps[at]) - kExpBias);
        vscale = pow2(int(P.value_exps[at]) - kExpBias);
      }
      if (s == -INFINITY) continue;  // weighs nothing beside any other score
      if (s > m + kAnyMove) {
        const float alpha = ex2(m - s);
        m = s;
        pl *= alpha;
#pragma unroll
        for (int k = 0; k < kAnyChunks; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) po[k][e] *= alpha;
      }
      const float p = ex2(s - m), pv = p * vscale;
      pl += p;
#pragma unroll
      for (int k = 0; k < kAnyChunks; ++k) {
        const int d = (lane + 32 * k) * 8;
        if (d >= P.hv) break;
        float x[8];
        widen8<Q8>(value[k], x);
#pragma unroll
        for (int e = 0; e < 8; ++e) po[k][e] += pv * x[e];
      }
    }
    const float alpha = m == m_folded ? 1.f : ex2(m_folded - m);
    m_folded = m;
    l *= alpha;
    l_lost *= alpha;
    add_two_sum(l, l_lost, pl);
#pragma unroll
    for (int k = 0; k < kAnyChunks; ++k) {
      const int d = (lane + 32 * k) * 8;
      if (d >= P.hv) break;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float sum = o_s[warp][d + e] * alpha, lost = lost_s[warp][d + e] * alpha;
        add_two_sum(sum, lost, po[k][e]);
        o_s[warp][d + e] = sum;
        lost_s[warp][d + e] = lost;
      }
    }
  }
  // (a sum that is no number lost none)
  if (isfinite(l)) l += l_lost;
#pragma unroll
  for (int k = 0; k < kAnyChunks; ++k) {
    const int d = (lane + 32 * k) * 8;
    if (d >= P.hv) break;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (isfinite(o_s[warp][d + e])) o_s[warp][d + e] += lost_s[warp][d + e];
  }
  if (lane == 0) {
    m_s[warp] = m;
    l_s[warp] = l;
  }
  __syncthreads();
  float M = m_s[0];
#pragma unroll
  for (int w = 1; w < kAnyWarps; ++w) M = fmaxf(M, m_s[w]);
  for (int d = threadIdx.x; d < P.hv; d += blockDim.x) {
    float sum = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kAnyWarps; ++w) {
      const float f = ex2(m_s[w] - M);
      sum += l_s[w] * f;
      acc += o_s[w][d] * f;
    }
    P.out[(t * P.num_heads + h) * P.hv + d] = __float2half_rn(acc / sum);
  }
}

}  // namespace pa
