// Tree attention over INT8 layers (kvq_tree.cuh).
#include "kvq_tree.cuh"

namespace kvq {

cudaError_t launch_tree_int8(const TreeParams& p, int nt, int ctas, int smem, cudaStream_t stream) {
  return launch_tree_fmt<KVQ_FMT_INT8>(p, nt, ctas, smem, stream);
}

}  // namespace kvq
