// Launch of the tcgen05 tree attention kernels (pa_tree_tc.cuh).
#include "pa_tree_tc_launch.cuh"

namespace pa {

cudaError_t tree_tc(const TreeParams& P, int head_size, bool q8, int64_t rows, int sms, size_t* need,
                    void* ws, cudaStream_t s) {
  if (tree_segments(P, rows > 128 ? 256 : 128)) return tree_tc_long(P, head_size, q8, rows, sms, need, ws, s);
  return head_size == 64 ? tree_tc_pick<64, false, false>(P, q8, rows, sms, need, ws, s)
                         : tree_tc_pick<128, false, false>(P, q8, rows, sms, need, ws, s);
}

}  // namespace pa
