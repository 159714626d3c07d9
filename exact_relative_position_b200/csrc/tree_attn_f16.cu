// tree_attn_f16.cu -- tree attention of fp16 queries over a cache in their own type.
#include "tree_attn.cuh"

namespace relpos {
namespace tree {
cudaError_t run_f16(const TreeParams& p, cudaStream_t s) { return run_format<__half, RELPOS_CACHE_F16>(p, s); }
}  // namespace tree
}  // namespace relpos
