// Attention with a sliding window and sinks over a paged cache (pa_window.h): the C entry
// and the choice of the kernel.
#include <cuda_runtime.h>

#include "pa_internal.h"
#include "pa_tree_any.cuh"
#include "pa_tree_host.h"
#include "pa_tree_tc.cuh"
#include "pa_window.h"

namespace pa {

namespace {

pa_status check_window(const pa_config* cfg, const pa_window* win) {
  const pa_status st = check_tree(cfg);
  if (st != PA_OK) return st;
  return win && win->window > 0 && win->sinks >= 0 ? PA_OK : PA_ERR_INVALID_ARG;
}

// The kernel for these head sizes and rows, if there is a faster one than tree_any_kernel: of 64 and 128 dims the
// tcgen05 tensor cores from 17 rows of a kv head on over the fp16 cache and from 33 on over the 8-bit
// one, else the warp-level tensor instructions with the least of 64, 128 and 256 dims that hold a head,
// in tiles of 8 rows or several of 16. 32 sequences, 8 kv heads of 128 dims, window 1024: 20 rows take 41 us here and
// 57 there in fp16, 53 and 43 in 8 bits; 32 rows 42 and 60, 53 and 46; 64 rows 44 and 107, 54 and 76.
// Window 4096: 20 rows 99 and 178 us, 105 and 108; 32 rows 100 and 184, 106 and 111. Of 64 dims, window
// 1024: 20 rows 34 and 36 us in fp16, 36 rows 34 and 45, and 46 and 50 in 8 bits. Sizes that the tcgen05 kernel does not
// have read the keys again for every 16 rows: prompts of 1024 to 8192 tokens, window 1024, take 3.5 ms at 256 dims
// (2.0 in 8 bits) and 2.4 at 96 (1.9).
// The rows are those of the longest sequence that the step allows, whatever the others are: 63 decode steps and a part
// of 512 tokens, window 2048, take 129 us in one call, 86 and 36 in two (fp16; 154, and 50 and 41 in 8 bits), so
// prompts' parts are better a call of their own.
bool window_tiles(const pa_config& c, const TreeParams& P, bool q8, size_t* need, void* ws, cudaStream_t stream,
                  cudaError_t* e) {
  const int hd = c.head_size_k > c.head_size_v ? c.head_size_k : c.head_size_v;
  const int64_t rows = int64_t(c.num_heads / c.kv_heads) * max_q(c);
  const int nt = rows <= 8 ? 1 : 2;
  if (rows > (q8 ? 32 : 16) && c.head_size_k == c.head_size_v && (hd == 64 || hd == 128))
    *e = window_tc(P, hd, q8, rows, c.num_sms, need, ws, stream);
  else if (hd <= 64)
    *e = window_mma_64(P, q8, nt, c.num_sms, need, ws, stream);
  else if (hd <= 128)
    *e = window_mma_128(P, q8, nt, c.num_sms, need, ws, stream);
  else if (hd <= 256)
    *e = window_mma_256(P, q8, nt, c.num_sms, need, ws, stream);
  else
    return false;
  return true;
}

}  // namespace

}  // namespace pa

extern "C" pa_status pa_window_workspace(const pa_config* cfg, const pa_window* win, size_t* workspace_bytes) {
  const pa_status st = pa::check_window(cfg, win);
  if (st != PA_OK) return st;
  if (!workspace_bytes) return PA_ERR_INVALID_ARG;
  // the larger of the two caches' needs, so that it does not depend on them
  *workspace_bytes = PA_STATUS_BYTES;
  pa::TreeParams P{};
  pa::tree_lengths(*cfg, P);
  P.window = win->window;
  P.sinks = win->sinks;
  for (const bool q8 : {false, true}) {
    size_t need = 0;
    cudaError_t e;
    if (pa::window_tiles(*cfg, P, q8, &need, nullptr, nullptr, &e) && need > *workspace_bytes)
      *workspace_bytes = need;
  }
  return PA_OK;
}

namespace pa {

namespace {

pa_status window_forward(const pa_config* cfg, const pa_window* win, int64_t tokens, const void* query,
                         const void* key_cache, const void* value_cache, const uint8_t* key_exps,
                         const uint8_t* value_exps, const int32_t* block_tables,
                         const int32_t* context_lens, const int32_t* q_seqlens, void* workspace,
                         size_t workspace_bytes, void* out, void* stream_) {
  size_t need = 0;
  pa_status st = pa_window_workspace(cfg, win, &need);
  if (st != PA_OK) return st;
  TreeParams P{};
  st = tree_arguments(*cfg, tokens, query, key_cache, value_cache, key_exps, value_exps, block_tables, context_lens,
                      q_seqlens, workspace, workspace_bytes, need, out, P);
  if (st != PA_OK || tokens == 0) return st;
  P.window = win->window;
  P.sinks = win->sinks;
  const cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  cudaError_t e = cudaSuccess;
  if (window_tiles(*cfg, P, key_exps != nullptr, nullptr, workspace, stream, &e))
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
  const unsigned grid = unsigned(tokens * cfg->num_heads);
  if (key_exps) tree_any_kernel<true, true><<<grid, kAnyWarps * 32, 0, stream>>>(P);
  else tree_any_kernel<false, true><<<grid, kAnyWarps * 32, 0, stream>>>(P);
  return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

}  // namespace pa

extern "C" pa_status pa_window_forward(const pa_config* cfg, const pa_window* win, int64_t tokens, const void* query,
                                       const void* key_cache, const void* value_cache, const uint8_t* key_exps,
                                       const uint8_t* value_exps, const int32_t* block_tables,
                                       const int32_t* context_lens, const int32_t* q_seqlens, void* workspace,
                                       size_t workspace_bytes, void* out, void* stream_) {
  try {
    return pa::window_forward(cfg, win, tokens, query, key_cache, value_cache, key_exps, value_exps, block_tables,
                              context_lens, q_seqlens, workspace, workspace_bytes, out, stream_);
  } catch (...) {  // of the host's memory or locks
    return PA_ERR_CUDA;
  }
}
