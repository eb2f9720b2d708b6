// What the kernels of pa_tree_forward and pa_window_forward share: their parameters, the lookup of a
// token's sequence, and the walk from a draft to its root.
#pragma once

#include "pa_device.cuh"
#include "pa_e4m3.cuh"
#include "pa_tree.h"

namespace pa {

// Cycles of a wait that has no other limit, about a second and a half: the 32-bit clock tells it.
constexpr uint32_t kTreeWaitLimit = 3u << 30;
constexpr int kTreeWords = PA_TREE_MAX_TOKENS / 32;  // ancestor bits of one draft

struct TreeParams {
  const __half* query;
  const uint8_t *key_cache, *value_cache;  // fp16 or e4m3 bytes
  const uint8_t *key_exps, *value_exps;
  const int32_t *block_tables, *context_lens, *q_seqlens, *parents;
  __half* out;
  uint32_t* status;
  int64_t tokens;
  int batch, num_heads, kv_heads, group, hk, hv, block_size, num_blocks, max_blocks_per_seq;
  int max_q, max_keys;
  int window, sinks;  // (pa_window_forward)
  uint32_t group_inverse;  // ceil(2^32 / group) where the group is below 2^15 and above 1, else 0
  float scale_log2;  // scale * log2(e)
  uint32_t wait_limit;  // cycles a wait on another role's progress may take
};

// The status bit of a length (no word is there to tell it to on the host, where tests run the division of the work).
__host__ __device__ __forceinline__ void tree_bad_length(const TreeParams& P) {
#ifdef __CUDA_ARCH__
  set_status(P.status, PA_STATUS_BIT_PLAN);
#endif
}

// Whether a sequence's lengths keep the constraints.
__host__ __device__ __forceinline__ bool tree_lengths_ok(const TreeParams& P, int q, int L) {
  return q >= 0 && q <= P.max_q && q <= P.tokens && L >= q && L <= P.max_keys;
}

// Whether a row is padding although it counts as one: without q_seqlens, that of a sequence without keys.
__host__ __device__ __forceinline__ bool tree_padding(const TreeParams& P, int L) { return !P.q_seqlens && L == 0; }

// Whether the tokens end before sequence rows begun at q_start do (the rows past them are left out).
__host__ __device__ __forceinline__ bool tree_rows_missing(const TreeParams& P, int q_start, int q) {
  return P.tokens - q_start < q;
}

// a + b tokens, at most all of them: where the rows of a sequence begin is a sum of the
// lengths before it, which may be any.
__host__ __device__ __forceinline__ int tree_tokens(const TreeParams& P, int a, int b) {
  return int(min(uint32_t(a) + uint32_t(b), uint32_t(P.tokens)));
}

// Sequence and index in it of token t (warp-collective); -1 past the last one.
// Every sequence counts with the length it states (a negative one with 0), whether
// it is valid or not: the rows lie as the lengths say.
__device__ __forceinline__ int tree_sequence(const TreeParams& P, int64_t t, int lane, int& index) {
  index = 0;
  if (!P.q_seqlens) return t < P.batch ? int(t) : -1;
  int before = 0;
  for (int b0 = 0; b0 < P.batch; b0 += 32) {
    int upto = b0 + lane < P.batch ? tree_tokens(P, 0, max(P.q_seqlens[b0 + lane], 0)) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto = tree_tokens(P, upto, up);
    }
    // the first lane whose sequence ends behind the token holds it
    const unsigned who = __ballot_sync(0xffffffffu, t - before < upto);
    if (who) {
      const int l = __ffs(who) - 1;
      const int start = __shfl_sync(0xffffffffu, upto, l > 0 ? l - 1 : 0);
      index = int(t - before) - (l > 0 ? start : 0);
      return b0 + l;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);  // at most t
  }
  return -1;
}

// Ancestor bits of draft i (itself among them) of the sequence whose parents
// begin at `parents`. A parent must come before its child, so the walk ends.
__device__ __forceinline__ void tree_ancestors(const TreeParams& P, const int32_t* parents, int i,
                                               uint32_t (&bits)[kTreeWords]) {
#pragma unroll
  for (int w = 0; w < kTreeWords; ++w) bits[w] = 0;
  while (true) {
    bits[i >> 5] |= 1u << (i & 31);
    const int up = parents[i];
    if (up < 0 || up >= i) {
      if (up != -1) set_status(P.status, PA_STATUS_BIT_TREE);
      return;
    }
    i = up;
  }
}

// Adds to one row's result what was taken out of its product: the non-finite
// elements of the values of the drafts flagged in `bad` (draft a under bit a
// modulo its size) that the row sees. `key0`, `key1` bound the keys that the result
// is of; `seen` are the row's ancestor bits, or null for a chain, whose row is draft
// `qi`. The result is fp16 (`out`) or an fp32 partial one (`part`, `stride`
// apart); dims first, first + step, ... below `last`. Rare, hence not inlined.
template <bool Q8>
__device__ __noinline__ void tree_patch(const TreeParams& P, int b, int q, int prefix, int kvh, int qi,
                                        const uint32_t* bad, const uint32_t* seen, int key0, int key1,
                                        __half* out, float* part, int stride, int first, int step, int last) {
  const int32_t* table = P.block_tables + int64_t(b) * P.max_blocks_per_seq;
  for (int a = max(key0 - prefix, 0); a < min(q, key1 - prefix); ++a) {
    if (!(bad[(a >> 5) % kTreeWords] >> (a & 31) & 1)) continue;
    if (seen ? !(seen[a >> 5] >> (a & 31) & 1) : a > qi) continue;
    const int key = prefix + a, block = table[key / P.block_size];
    if (block < 0 || block >= P.num_blocks) continue;
    const int64_t row = ((int64_t(block) * P.block_size + key % P.block_size) * P.kv_heads + kvh) * P.hv;
    for (int d = first; d < last; d += step) {
      const float v = Q8 ? h2f2(e4m3x2_half2(P.value_cache[row + d])).x
                         : __half2float(*reinterpret_cast<const __half*>(P.value_cache + 2 * (row + d)));
      if (isfinite(v)) continue;
      if (out) out[d] = __float2half_rn(__half2float(out[d]) + v);
      else part[int64_t(d) * stride] += v;
    }
  }
}

}  // namespace pa
