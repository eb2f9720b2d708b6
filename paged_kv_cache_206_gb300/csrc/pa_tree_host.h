// Host side that pa_tree_forward and pa_window_forward share: the checks of a call and the
// parameters of its kernels.
#pragma once

#include <algorithm>
#include <cmath>

#include "pa_internal.h"
#include "pa_tree.cuh"

namespace pa {

inline pa_status check_tree(const pa_config* cfg) {
  const pa_status st = validate_config(cfg);
  if (st != PA_OK) return st;
  if (cfg->mask_type != PA_MASK_NONE || cfg->chunk_blocks != 0 || cfg->num_sms <= 0 ||
      cfg->num_sms > 65535)
    return PA_ERR_INVALID_ARG;
  return PA_OK;
}

inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// The longest context. The kernels count keys in 32 bits, and units of keys and what a row tile costs besides
// past a context's end.
constexpr int64_t kMostKeys = (int64_t(1) << 31) - 4096;

// What of P says how long a tile may be: all that a workspace's size asks of it.
inline void tree_lengths(const pa_config& c, TreeParams& P) {
  P.max_keys = int(std::min<int64_t>(int64_t(c.max_blocks_per_seq) * c.block_size, kMostKeys));
}

// The checks behind check_tree, and P of the arguments (of no tokens: nothing).
inline pa_status tree_arguments(const pa_config& c, int64_t tokens, const void* query, const void* key_cache,
                                const void* value_cache, const uint8_t* key_exps, const uint8_t* value_exps,
                                const int32_t* block_tables, const int32_t* context_lens, const int32_t* q_seqlens,
                                void* workspace, size_t workspace_bytes, size_t need, void* out, TreeParams& P) {
  if (tokens < 0 || !query || !key_cache || !value_cache || !block_tables || !context_lens ||
      !workspace || !out || (key_exps == nullptr) != (value_exps == nullptr))
    return PA_ERR_INVALID_ARG;
  if (key_cache == value_cache || (key_exps && key_exps == value_exps)) return PA_ERR_INVALID_ARG;
  if (!aligned(query, 16) || !aligned(key_cache, 16) || !aligned(value_cache, 16) ||
      !aligned(key_exps, 16) || !aligned(value_exps, 16) || !aligned(out, 16) ||
      !aligned(workspace, 256))
    return PA_ERR_INVALID_ARG;
  if (workspace_bytes < need) return PA_ERR_BUFFER_TOO_SMALL;
  if (tokens > INT32_MAX / c.num_heads) return PA_ERR_INVALID_ARG;
  if (tokens == 0) return PA_OK;
  if (out == query) return PA_ERR_INVALID_ARG;  // a tile in parts reads its rows after others wrote theirs
  P.query = static_cast<const __half*>(query);
  P.key_cache = static_cast<const uint8_t*>(key_cache);
  P.value_cache = static_cast<const uint8_t*>(value_cache);
  P.key_exps = key_exps;
  P.value_exps = value_exps;
  P.block_tables = block_tables;
  P.context_lens = context_lens;
  P.q_seqlens = q_seqlens;
  P.out = static_cast<__half*>(out);
  P.status = static_cast<uint32_t*>(workspace);
  P.tokens = tokens;
  P.batch = c.batch;
  P.num_heads = c.num_heads;
  P.kv_heads = c.kv_heads;
  P.group = c.num_heads / c.kv_heads;
  P.group_inverse = P.group > 1 && P.group < (1 << 15) ? uint32_t((uint64_t(1) << 32) / P.group + 1) : 0;
  P.hk = c.head_size_k;
  P.hv = c.head_size_v;
  P.block_size = c.block_size;
  P.num_blocks = c.num_blocks;
  P.max_blocks_per_seq = c.max_blocks_per_seq;
  P.max_q = int(max_q(c));
  tree_lengths(c, P);
  P.scale_log2 = (c.scale > 0.f ? c.scale : 1.0f / std::sqrt(float(c.head_size_k))) * kLog2e;
  P.wait_limit = uint32_t(std::min<long long>(wait_limit(), kTreeWaitLimit));
  return PA_OK;
}

}  // namespace pa
