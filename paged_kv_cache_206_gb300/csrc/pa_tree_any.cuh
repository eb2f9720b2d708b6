// The attention kernel of pa_tree_forward and pa_window_forward for the largest heads.
#pragma once

#include "pa_tree.cuh"

namespace pa {

constexpr int kAnyWarps = 4;
constexpr int kAnyChunks = (PA_MAX_HEAD_SIZE / 8 + 31) / 32;  // 8-dim chunks a lane may hold

// 8 elements of a cache row as fp32.
template <bool Q8>
__device__ __forceinline__ void load8(const uint8_t* row, int d, float (&x)[8]) {
  uint32_t h[4];
  if constexpr (Q8) {
    const uint2 c = *reinterpret_cast<const uint2*>(row + d);
    h[0] = e4m3x2_half2(c.x);
    h[1] = e4m3x2_half2(c.x >> 16);
    h[2] = e4m3x2_half2(c.y);
    h[3] = e4m3x2_half2(c.y >> 16);
  } else {
    const uint4 c = *reinterpret_cast<const uint4*>(row + 2 * d);
    h[0] = c.x;
    h[1] = c.y;
    h[2] = c.z;
    h[3] = c.w;
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
    if (!tree_lengths_ok(P, q, P.context_lens[b])) set_status(P.status, PA_STATUS_BIT_PLAN);
    sum += max(q, 0);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (sum > P.tokens) set_status(P.status, PA_STATUS_BIT_PLAN);
}

// Heads of more than 256 dims. One CTA per (token, head); warp w takes the keys w, w + 4,
// ..., a lane holds 8-dim chunks lane, lane + 32, ... of the row. Softmax and sums in fp32.
// Bound by the latency of a key after another, and the heads of a group read the
// same keys each: 2.4 ms for 64 decode steps of up to 4096 keys of 8 kv heads, whatever
// their size. WIN: the keys are the sinks before the window, then those of the window.
template <bool Q8, bool WIN>
__global__ void __launch_bounds__(kAnyWarps * 32) tree_any_kernel(const TreeParams P) {
  __shared__ float o_s[kAnyWarps][PA_MAX_HEAD_SIZE];
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
    set_status(P.status, PA_STATUS_BIT_PLAN);
    return;
  }
  const int prefix = L - q;
  uint32_t bits[kTreeWords];
  if (!WIN && P.parents) tree_ancestors(P, P.parents + (t - i), i, bits);

  float query[kAnyChunks][8], o[kAnyChunks][8];
#pragma unroll
  for (int k = 0; k < kAnyChunks; ++k) {
    const int d = (lane + 32 * k) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) query[k][j] = o[k][j] = 0.f;
    if (d < P.hk)
      load8<false>(reinterpret_cast<const uint8_t*>(P.query + (t * P.num_heads + h) * P.hk), d, query[k]);
  }
  float m = -INFINITY, l = 0.f;
  const int lo = WIN ? max(prefix + i - P.window + 1, 0) : 0, far = WIN ? min(P.sinks, lo) : 0;
  const int keys = prefix + i + 1 - (lo - far);
  for (int n = warp; n < keys; n += kAnyWarps) {
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
    float dot = 0.f;
#pragma unroll
    for (int k = 0; k < kAnyChunks; ++k) {
      const int d = (lane + 32 * k) * 8;
      if (d >= P.hk) break;
      float x[8];
      load8<Q8>(kr, d, x);
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
    const float mn = fmaxf(m, s), alpha = ex2(m - mn), p = ex2(s - mn), pv = p * vscale;
    m = mn;
    l = l * alpha + p;
    const uint8_t* vr = P.value_cache + row * P.hv * (Q8 ? 1 : 2);
#pragma unroll
    for (int k = 0; k < kAnyChunks; ++k) {
      const int d = (lane + 32 * k) * 8;
      if (d >= P.hv) break;
      float x[8];
      load8<Q8>(vr, d, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[k][e] = o[k][e] * alpha + pv * x[e];
    }
  }
#pragma unroll
  for (int k = 0; k < kAnyChunks; ++k) {
    const int d = (lane + 32 * k) * 8;
    if (d >= P.hv) break;
#pragma unroll
    for (int e = 0; e < 8; ++e) o_s[warp][d + e] = o[k][e];
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
