// Tree attention over FP8 E4M3 layers (kvq_tree.cuh).
#include "kvq_tree.cuh"

namespace kvq {

size_t tree_fixed_smem(int nt, int batch) {
  const size_t big = nt == 32 ? TreeShape<32>::kFixed : (nt == 64 ? TreeShape<64>::kFixed : TreeShape<128>::kFixed);
  return 1024 + big + sizeof(TreeSmem) + (3 * (size_t)batch + 1) * sizeof(int);  // (1024: alignment of the base)
}

cudaError_t launch_tree_fp8(const TreeParams& p, int nt, int ctas, int smem, cudaStream_t stream) {
  return launch_tree_fmt<KVQ_FMT_FP8_E4M3>(p, nt, ctas, smem, stream);
}

}  // namespace kvq
