// The same as pa_tree_tc.cu for tiles that may be taken in segments (pa_tree_split.cuh).
#include "pa_tree_tc_launch.cuh"

namespace pa {

cudaError_t tree_tc_long(const TreeParams& P, int head_size, bool q8, int64_t rows, int sms, size_t* need,
                         void* ws, cudaStream_t s) {
  return head_size == 64 ? tree_tc_pick<64, false, true>(P, q8, rows, sms, need, ws, s)
                         : tree_tc_pick<128, false, true>(P, q8, rows, sms, need, ws, s);
}

}  // namespace pa
