// Tree attention over INT2 layers (kvq_tree.cuh).
#include "kvq_tree.cuh"

namespace kvq {

cudaError_t launch_tree_int2(const TreeParams& p, int nt, int ctas, int smem, cudaStream_t stream) {
  return launch_tree_fmt<KVQ_FMT_INT2>(p, nt, ctas, smem, stream);
}

}  // namespace kvq
