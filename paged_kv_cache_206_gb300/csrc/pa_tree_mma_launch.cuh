// Host side of pa_tree_mma.cuh, included by one source file per head size.
#pragma once

#include "pa_internal.h"
#include "pa_launch.h"
#include "pa_tree_mma.cuh"

namespace pa {

// A cache as (bytes of a row, kv heads, token rows), a box being up to 128 bytes of
// `box` tokens of one head, swizzled, zeros behind a row's end.
inline bool tree_rows_map(CUtensorMap* m, const void* base, const TreeParams& P, int row_bytes, int part, int box) {
  const cuuint64_t dims[3] = {cuuint64_t(row_bytes), cuuint64_t(P.kv_heads),
                              cuuint64_t(P.num_blocks) * P.block_size};
  const cuuint64_t strides[2] = {cuuint64_t(row_bytes), cuuint64_t(P.kv_heads) * row_bytes};
  const cuuint32_t b[3] = {cuuint32_t(part), 1, cuuint32_t(box)}, es[3] = {1, 1, 1};
  return encode_tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, b, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, part == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

template <int HD, bool Q8, int NT>
cudaError_t tree_mma_run(const TreeParams& P, int sms, size_t* need, void* ws, cudaStream_t stream) {
  using Cfg = TreeMma<HD, Q8, NT>;
  const int grid = sms * Cfg::kCtas, workers = grid * Cfg::kWarps;
  const size_t rows = size_t(2) * workers * Cfg::kRows;
  const size_t o_off = PA_STATUS_BYTES, ml_off = align256(o_off + rows * HD * 4);
  const size_t join_off = align256(ml_off + rows * sizeof(float2));
  if (need) {
    *need = align256(join_off + workers * sizeof(TreeJoin));
    return cudaSuccess;
  }
  TreeSplit S;
  S.part_o = reinterpret_cast<float*>(static_cast<char*>(ws) + o_off);
  S.part_ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + ml_off);
  S.join = reinterpret_cast<TreeJoin*>(static_cast<char*>(ws) + join_off);
  S.workers = workers;
  // a partial result (kRows rows of fp32) should stay below the keys it stands for
  S.min_units = Cfg::kLead + (NT + Cfg::kMT - 1) / Cfg::kMT;
  auto kern = tree_mma_kernel<HD, Q8, NT>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), Cfg::bytes);
  if (e != cudaSuccess) return e;
  const int low = P.block_size & -P.block_size, box = low < Cfg::kSub ? low : Cfg::kSub;
  CUtensorMap tmk, tmv;
  const int part = Cfg::kRowBytes < 128 ? Cfg::kRowBytes : 128, elem = Q8 ? 1 : 2;
  if (!tree_rows_map(&tmk, P.key_cache, P, P.hk * elem, part, box) ||
      !tree_rows_map(&tmv, P.value_cache, P, P.hv * elem, part, box))
    return cudaErrorInvalidValue;
  kern<<<unsigned(grid), Cfg::kWarps * 32, Cfg::bytes, stream>>>(tmk, tmv, P, S, box);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(workers), NT);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_combine_kernel<HD, Cfg::kRows>, P, S);
}

template <int HD>
cudaError_t tree_mma_pick(const TreeParams& P, bool q8, int nt, int sms, size_t* need, void* ws,
                          cudaStream_t s) {
  if (nt >= 2)
    return q8 ? tree_mma_run<HD, true, 2>(P, sms, need, ws, s) : tree_mma_run<HD, false, 2>(P, sms, need, ws, s);
  return q8 ? tree_mma_run<HD, true, 1>(P, sms, need, ws, s) : tree_mma_run<HD, false, 1>(P, sms, need, ws, s);
}

}  // namespace pa
