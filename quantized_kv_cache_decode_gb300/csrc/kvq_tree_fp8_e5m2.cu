// Tree attention over FP8 E5M2 layers (kvq_tree.cuh).
#include "kvq_tree.cuh"

namespace kvq {

cudaError_t launch_tree_fp8_e5m2(const TreeParams& p, int nt, int ctas, int smem, cudaStream_t stream) {
  return launch_tree_fmt<KVQ_FMT_FP8_E5M2>(p, nt, ctas, smem, stream);
}

}  // namespace kvq
