// The warp-level tree attention kernels for heads of up to 64 dims (pa_tree_mma.cuh).
#include "pa_tree_mma_launch.cuh"

namespace pa {

cudaError_t tree_mma_64(const TreeParams& P, bool q8, int nt, int sms, size_t* need, void* ws,
                        cudaStream_t s) {
  if (tree_segments(P, 8 * nt)) return tree_mma_long_64(P, q8, nt, sms, need, ws, s);
  return tree_mma_pick<64, false, false>(P, q8, nt, sms, need, ws, s);
}

}  // namespace pa
