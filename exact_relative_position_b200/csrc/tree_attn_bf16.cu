// tree_attn_bf16.cu -- tree attention of bf16 queries over a cache in their own type.
#include "tree_attn.cuh"

namespace relpos {
namespace tree {
cudaError_t run_bf16(const TreeParams& p, cudaStream_t s) { return run_format<__nv_bfloat16, RELPOS_CACHE_F16>(p, s); }
}  // namespace tree
}  // namespace relpos
