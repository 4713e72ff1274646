// Tree attention over FP8 E4M3 layers (kvq_tree.cuh).
#include "kvq_tree.cuh"

namespace kvq {

size_t tree_fixed_smem(int sub, int batch) {
  const size_t big = sub == 16 ? TreeShape<16>::kFixed : (sub == 32 ? TreeShape<32>::kFixed : TreeShape<64>::kFixed);
  return 1024 + big + sizeof(TreeSmem) + (2 * (size_t)batch + 1) * sizeof(int);  // (1024: alignment of the base)
}

cudaError_t launch_tree_fp8(const TreeParams& p, int sub, int ctas, int smem, cudaStream_t stream) {
  return launch_tree_fmt<KVQ_FMT_FP8_E4M3>(p, sub, ctas, smem, stream);
}

}  // namespace kvq
