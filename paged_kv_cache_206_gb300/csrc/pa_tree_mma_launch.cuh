// Host side of pa_tree_mma.cuh, included by one source file per head size.
#pragma once

#include "pa_internal.h"
#include "pa_launch.h"
#include "pa_tree_mma.cuh"

namespace pa {

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
  kern<<<unsigned(grid), Cfg::kWarps * 32, Cfg::bytes, stream>>>(P, S);
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
