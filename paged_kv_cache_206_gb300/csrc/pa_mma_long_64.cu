// The same as pa_tree_mma_64.cu and pa_window_mma_64.cu for tiles that may be taken in segments (pa_tree_split.cuh).
#include "pa_tree_mma_launch.cuh"

namespace pa {

cudaError_t tree_mma_long_64(const TreeParams& P, bool q8, int nt, int sms, size_t* need, void* ws, cudaStream_t s) {
  return tree_mma_pick<64, false, true>(P, q8, nt, sms, need, ws, s);
}
cudaError_t window_mma_long_64(const TreeParams& P, bool q8, int nt, int sms, size_t* need, void* ws, cudaStream_t s) {
  return tree_mma_pick<64, true, true>(P, q8, nt, sms, need, ws, s);
}

}  // namespace pa
