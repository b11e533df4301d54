// Attention over the paged cache (tree_attention.cuh): bf16, 64 dimensions.
#include "tree_attention.cuh"

namespace idx {

cudaError_t launch_tree_attention_bf16_64(const TreeAttnArgs &a, const CUtensorMap &qm, const CUtensorMap &km,
                                       const CUtensorMap &vm, int num_ctas, cudaStream_t stream) {
  return a.sel != nullptr ? launch_shape<64, false, true>(a, qm, km, vm, num_ctas, stream)
                          : launch_shape<64, false, false>(a, qm, km, vm, num_ctas, stream);
}

}  // namespace idx
