// Attention for drafted tokens over a paged cache (pa_tree.h): the C entry, the
// choice of the kernel.
#include <cuda_runtime.h>

#include "pa_internal.h"
#include "pa_tree_any.cuh"
#include "pa_tree_host.h"
#include "pa_tree_tc.cuh"

namespace pa {

namespace {

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

}  // namespace

}  // namespace pa

extern "C" pa_status pa_tree_workspace(const pa_config* cfg, size_t* workspace_bytes) {
  const pa_status st = pa::check_tree(cfg);
  if (st != PA_OK) return st;
  if (!workspace_bytes) return PA_ERR_INVALID_ARG;
  // the larger of the two caches' needs, so that it does not depend on them
  *workspace_bytes = PA_STATUS_BYTES;
  pa::TreeParams P{};
  pa::tree_lengths(*cfg, P);
  for (const bool q8 : {false, true}) {
    size_t need = 0;
    cudaError_t e;
    if (pa::tree_tiles(*cfg, P, q8, &need, nullptr, nullptr, &e) && need > *workspace_bytes)
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
  pa_status st = pa_tree_workspace(cfg, &need);
  if (st != PA_OK) return st;
  if (parents && max_q(*cfg) > PA_TREE_MAX_TOKENS) return PA_ERR_INVALID_ARG;
  TreeParams P{};
  st = tree_arguments(*cfg, tokens, query, key_cache, value_cache, key_exps, value_exps, block_tables, context_lens,
                      q_seqlens, workspace, workspace_bytes, need, out, P);
  if (st != PA_OK || tokens == 0) return st;
  P.parents = parents;
  const pa_config& c = *cfg;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  cudaError_t e = cudaSuccess;
  if (tree_tiles(c, P, key_exps != nullptr, nullptr, workspace, stream, &e))
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
  const unsigned grid = unsigned(tokens * c.num_heads);
  if (key_exps) tree_any_kernel<true, false><<<grid, kAnyWarps * 32, 0, stream>>>(P);
  else tree_any_kernel<false, false><<<grid, kAnyWarps * 32, 0, stream>>>(P);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}
