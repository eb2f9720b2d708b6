// Attention for drafted tokens over a paged cache (pa_tree.h): the C entry, the
// choice of the kernel, and the kernel for the largest heads.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "pa_internal.h"
#include "pa_tree_tc.cuh"

namespace pa {

namespace {

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
__device__ __noinline__ void tree_check_lengths(const TreeParams& P, int lane) {
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
// their size.
template <bool Q8>
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
  if (P.parents) tree_ancestors(P, P.parents + (t - i), i, bits);

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
  for (int j = warp; j <= prefix + i; j += kAnyWarps) {
    if (P.parents && j >= prefix) {
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

pa_status check_tree(const pa_config* cfg) {
  const pa_status st = validate_config(cfg);
  if (st != PA_OK) return st;
  if (cfg->mask_type != PA_MASK_NONE || cfg->chunk_blocks != 0 || cfg->num_sms <= 0 ||
      cfg->num_sms > 65535)
    return PA_ERR_INVALID_ARG;
  return PA_OK;
}

// The kernel for these head sizes and rows, if there is a faster one than
// tree_any_kernel: for up to 16 rows of a kv head the warp-level tensor instructions
// with the narrower of their 8- and 16-row tiles that holds the rows, and the least
// of 64, 128 and 256 dims that hold a head; for more rows of 64 or 128 dims the tcgen05
// tensor cores, of other sizes several of the 16-row tiles. Of 64 sequences of up to
// 4096 keys, 8 kv heads of 128 dims, 16 rows take 60 us (8 bits) and 89 us (fp16) here and
// 91 and 84 us there; one sequence of 1024 keys 19 and 18 us here, 21 and 16 us there. With
// 32 rows the warp-level instructions take 104 and 164 us (20 and 18 us for the one
// sequence), the others 93 and 86 us (22 and 16 us).
bool tree_tiles(const pa_config& c, const TreeParams& P, bool q8, size_t* need, void* ws,
                cudaStream_t stream, cudaError_t* e) {
  const int hd = c.head_size_k > c.head_size_v ? c.head_size_k : c.head_size_v;
  const int64_t rows = int64_t(c.num_heads / c.kv_heads) * max_q(c);
  const int nt = rows <= 8 ? 1 : 2;
  if (rows > 16 && c.head_size_k == c.head_size_v && (hd == 64 || hd == 128))
    *e = tree_tc(P, hd, q8, rows, c.num_sms, need, ws, stream);
  else if (hd <= 64)
    *e = tree_mma_64(P, q8, nt, c.num_sms, need, ws, stream);
  else if (hd <= 128)
    *e = tree_mma_128(P, q8, nt, c.num_sms, need, ws, stream);
  else if (hd <= 256)
    *e = tree_mma_256(P, q8, nt, c.num_sms, need, ws, stream);
  else
    return false;
  return true;
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace

}  // namespace pa

extern "C" pa_status pa_tree_workspace(const pa_config* cfg, size_t* workspace_bytes) {
  const pa_status st = pa::check_tree(cfg);
  if (st != PA_OK) return st;
  if (!workspace_bytes) return PA_ERR_INVALID_ARG;
  // the larger of the two caches' needs, so that it does not depend on them
  *workspace_bytes = PA_STATUS_BYTES;
  for (const bool q8 : {false, true}) {
    size_t need = 0;
    cudaError_t e;
    if (pa::tree_tiles(*cfg, pa::TreeParams{}, q8, &need, nullptr, nullptr, &e) && need > *workspace_bytes)
      *workspace_bytes = need;
  }
  return PA_OK;
}

extern "C" pa_status pa_tree_forward(const pa_config* cfg, int64_t tokens, const void* query,
                                     const void* key_cache, const void* value_cache,
                                     const uint8_t* key_exps, const uint8_t* value_exps,
                                     const int32_t* block_tables, const int32_t* context_lens,
                                     const int32_t* q_seqlens, const int32_t* parents,
                                     void* workspace, size_t workspace_bytes, void* out,
                                     void* stream_) {
  using namespace pa;
  size_t need = 0;
  const pa_status st = pa_tree_workspace(cfg, &need);
  if (st != PA_OK) return st;
  const pa_config& c = *cfg;
  if (tokens < 0 || !query || !key_cache || !value_cache || !block_tables || !context_lens ||
      !workspace || !out || (key_exps == nullptr) != (value_exps == nullptr))
    return PA_ERR_INVALID_ARG;
  if (key_cache == value_cache || (key_exps && key_exps == value_exps)) return PA_ERR_INVALID_ARG;
  if (parents && max_q(c) > PA_TREE_MAX_TOKENS) return PA_ERR_INVALID_ARG;
  if (!aligned(query, 16) || !aligned(key_cache, 16) || !aligned(value_cache, 16) ||
      !aligned(key_exps, 16) || !aligned(value_exps, 16) || !aligned(out, 16) ||
      !aligned(workspace, 256))
    return PA_ERR_INVALID_ARG;
  if (workspace_bytes < need) return PA_ERR_BUFFER_TOO_SMALL;
  if (tokens > INT32_MAX / c.num_heads) return PA_ERR_INVALID_ARG;
  if (tokens == 0) return PA_OK;
  if (out == query) return PA_ERR_INVALID_ARG;  // a tile in parts reads its rows after others wrote theirs
  TreeParams P{};
  P.query = static_cast<const __half*>(query);
  P.key_cache = static_cast<const uint8_t*>(key_cache);
  P.value_cache = static_cast<const uint8_t*>(value_cache);
  P.key_exps = key_exps;
  P.value_exps = value_exps;
  P.block_tables = block_tables;
  P.context_lens = context_lens;
  P.q_seqlens = q_seqlens;
  P.parents = parents;
  P.out = static_cast<__half*>(out);
  P.status = static_cast<uint32_t*>(workspace);
  P.tokens = tokens;
  P.batch = c.batch;
  P.num_heads = c.num_heads;
  P.kv_heads = c.kv_heads;
  P.group = c.num_heads / c.kv_heads;
  P.hk = c.head_size_k;
  P.hv = c.head_size_v;
  P.block_size = c.block_size;
  P.num_blocks = c.num_blocks;
  P.max_blocks_per_seq = c.max_blocks_per_seq;
  P.max_q = int(max_q(c));
  P.scale_log2 = (c.scale > 0.f ? c.scale : 1.0f / std::sqrt(float(c.head_size_k))) * kLog2e;
  P.wait_limit = uint32_t(std::min<long long>(wait_limit(), kTreeWaitLimit));
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  cudaError_t e = cudaSuccess;
  if (tree_tiles(c, P, key_exps != nullptr, nullptr, workspace, stream, &e))
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
  const unsigned grid = unsigned(tokens * c.num_heads);
  if (key_exps) tree_any_kernel<true><<<grid, kAnyWarps * 32, 0, stream>>>(P);
  else tree_any_kernel<false><<<grid, kAnyWarps * 32, 0, stream>>>(P);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
