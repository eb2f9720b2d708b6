// The warp-level tree attention kernels for heads of up to 256 dims (pa_tree_mma.cuh).
#include "pa_tree_mma_launch.cuh"

namespace pa {

cudaError_t tree_mma_256(const TreeParams& P, bool q8, int nt, int sms, size_t* need, void* ws,
                        cudaStream_t s) {
  return tree_mma_pick<256>(P, q8, nt, sms, need, ws, s);
}

}  // namespace pa
