// Attention over the paged cache with few rows (tree_attention_few.cuh): bf16, 64 dimensions.
#include "tree_attention_few.cuh"

namespace idx {

cudaError_t launch_tree_few_bf16_64(const TreeAttnArgs &a, const CUtensorMap &qm, const CUtensorMap &km,
                                 const CUtensorMap &vm, int num_ctas, cudaStream_t stream) {
  const bool sel = a.sel != nullptr;
  if (a.rows == 16)
    return sel ? launch_few_rows<64, false, 16, true>(a, qm, km, vm, num_ctas, stream)
               : launch_few_rows<64, false, 16, false>(a, qm, km, vm, num_ctas, stream);
  if (a.rows == 32)
    return sel ? launch_few_rows<64, false, 32, true>(a, qm, km, vm, num_ctas, stream)
               : launch_few_rows<64, false, 32, false>(a, qm, km, vm, num_ctas, stream);
  return launch_few_rows<64, false, 64, true>(a, qm, km, vm, num_ctas, stream);   // 64 rows: selected only
}

}  // namespace idx
