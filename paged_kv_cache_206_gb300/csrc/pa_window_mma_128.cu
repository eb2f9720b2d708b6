// The warp-level attention kernels with a window for heads of up to 128 dims (pa_tree_mma.cuh).
#include "pa_tree_mma_launch.cuh"

namespace pa {

cudaError_t window_mma_128(const TreeParams& P, bool q8, int nt, int sms, size_t* need, void* ws,
                        cudaStream_t s) {
  if (tree_segments(P, 8 * nt)) return window_mma_long_128(P, q8, nt, sms, need, ws, s);
  return tree_mma_pick<128, true, false>(P, q8, nt, sms, need, ws, s);
}

}  // namespace pa
