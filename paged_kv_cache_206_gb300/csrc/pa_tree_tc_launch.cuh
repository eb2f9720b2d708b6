// Host side of pa_tree_tc.cuh, included by a source file for each kind of call.
#pragma once

#include <algorithm>

#include "pa_internal.h"
#include "pa_launch.h"
#include "pa_tree_tc.cuh"

namespace pa {

// The fp16 cache as (64 elements, token rows, 64-dim blocks of all kv heads), a box
// being `box` tokens of one block with the 128-byte swizzle; the 8-bit cache as
// (bytes of a row, token rows), a box being `box` tokens of one head.
inline bool tree_map(CUtensorMap* m, const void* base, const TreeParams& P, bool q8, int box) {
  const cuuint64_t rows = cuuint64_t(P.num_blocks) * P.block_size;
  const cuuint32_t es[3] = {1, 1, 1};
  if (q8) {
    const cuuint64_t dims[2] = {cuuint64_t(P.kv_heads) * P.hk, rows}, strides[1] = {dims[0]};
    const cuuint32_t b[2] = {cuuint32_t(P.hk), cuuint32_t(box)};
    return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, b, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  }
  const cuuint64_t dims[3] = {64, rows, cuuint64_t(P.kv_heads) * (P.hk / 64)};
  const cuuint64_t strides[2] = {cuuint64_t(P.kv_heads) * P.hk * 2, 128};
  const cuuint32_t b[3] = {64, cuuint32_t(box), 1};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, b, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

// The queries as (dims, heads, tokens), a box being 64 dims of a kv head's heads of as many tokens
// as make 128 rows.
inline bool window_query_map(CUtensorMap* m, const TreeParams& P) {
  const cuuint64_t dims[3] = {cuuint64_t(P.hk), cuuint64_t(P.num_heads), cuuint64_t(P.tokens)};
  const cuuint64_t strides[2] = {cuuint64_t(P.hk) * 2, cuuint64_t(P.num_heads) * P.hk * 2};
  const cuuint32_t b[3] = {64, cuuint32_t(P.group), cuuint32_t(128 / P.group)}, es[3] = {1, 1, 1};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<__half*>(P.query), dims, strides, b, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

template <int HD, bool Q8, int QT, bool WIN, bool SEG>
cudaError_t tree_tc_run(const TreeParams& P, int sms, size_t* need, void* ws, cudaStream_t stream) {
  using Cfg = TreeTc<HD, Q8, QT, WIN, SEG>;
  const size_t rows = size_t(SEG ? 3 : 2) * sms * Cfg::kRows;
  const size_t o_off = PA_STATUS_BYTES, ml_off = align256(o_off + rows * HD * 4);
  const size_t join_off = align256(ml_off + rows * sizeof(float2));
  const size_t fold_off = align256(join_off + sms * sizeof(TreeJoin));
  if (need) {
    *need = align256(fold_off + (SEG ? 2 * size_t(sms) * Cfg::kRows * sizeof(float2) : 0));
    return cudaSuccess;
  }
  TreeSplit S;
  S.part_o = reinterpret_cast<float*>(static_cast<char*>(ws) + o_off);
  S.part_ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + ml_off);
  S.join = reinterpret_cast<TreeJoin*>(static_cast<char*>(ws) + join_off);
  S.tile_tokens = std::max(Cfg::kRows / P.group, 1);
  S.tile_parts = (P.group - 1) / Cfg::kRows + 1;
  S.fold_ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + fold_off);
  S.workers = sms;
  S.segment = SEG ? kSegmentKeys / Cfg::kTok : 0;
  S.min_units = (Cfg::kLead + 1) * (WIN ? Cfg::kTok : 1);
  const int box = std::min(P.block_size & -P.block_size, 64);
  CUtensorMap tmk, tmv;
  if (!tree_map(&tmk, P.key_cache, P, Q8, box) || !tree_map(&tmv, P.value_cache, P, Q8, box))
    return cudaErrorInvalidValue;
  std::conditional_t<WIN, CUtensorMap, int> tmq{};
  if constexpr (WIN)
    if (128 % P.group == 0 && !window_query_map(&tmq, P)) return cudaErrorInvalidValue;
  auto kern = tree_tc_kernel<HD, Q8, QT, WIN, SEG>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), Cfg::bytes);
  if (e != cudaSuccess) return e;
  kern<<<unsigned(sms), Cfg::kThreads, Cfg::bytes, stream>>>(tmk, tmv, tmq, P, S);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(sms), Cfg::kRows / 32);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_combine_cols_kernel<HD, Cfg::kRows>, P, S);
}

template <int HD, bool WIN, bool SEG>
cudaError_t tree_tc_pick(const TreeParams& P, bool q8, int64_t rows, int sms, size_t* need, void* ws,
                 cudaStream_t s) {
  if (rows > 128)
    return q8 ? tree_tc_run<HD, true, 2, WIN, SEG>(P, sms, need, ws, s)
              : tree_tc_run<HD, false, 2, WIN, SEG>(P, sms, need, ws, s);
  return q8 ? tree_tc_run<HD, true, 1, WIN, SEG>(P, sms, need, ws, s)
            : tree_tc_run<HD, false, 1, WIN, SEG>(P, sms, need, ws, s);
}

}  // namespace pa
