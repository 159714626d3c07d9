// tree_attn_e4m3_bf16.cu -- tree attention of bf16 queries over an e4m3 cache.
#include "tree_attn.cuh"

namespace relpos {
namespace tree {
cudaError_t run_e4m3_bf16(const TreeParams& p, cudaStream_t s) { return run_format<__nv_bfloat16, RELPOS_CACHE_E4M3>(p, s); }
}  // namespace tree
}  // namespace relpos
