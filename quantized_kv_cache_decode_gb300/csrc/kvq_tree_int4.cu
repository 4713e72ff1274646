// Tree attention over INT4 layers (kvq_tree.cuh); bf16 layers run this instantiation (their blocks are all bf16 rows).
#include "kvq_tree.cuh"

namespace kvq {

cudaError_t launch_tree_int4(const TreeParams& p, int nt, int ctas, int smem, cudaStream_t stream) {
  return launch_tree_fmt<KVQ_FMT_INT4>(p, nt, ctas, smem, stream);
}

}  // namespace kvq
