// Attention over the paged cache with many rows (tree_attention_many.cuh): E4M3, 128 dimensions.
#include "tree_attention_many.cuh"

namespace idx {

cudaError_t launch_tree_many_e4m3_128(const TreeAttnArgs &a, const CUtensorMap &qm, const CUtensorMap &km,
                                  const CUtensorMap &vm, int num_ctas, cudaStream_t stream) {
  if (a.sel != nullptr) return launch<128, true, false, true>(a, qm, km, vm, num_ctas, stream);
  return a.pair ? launch<128, true, true, false>(a, qm, km, vm, num_ctas, stream)
                : launch<128, true, false, false>(a, qm, km, vm, num_ctas, stream);
}

}  // namespace idx
