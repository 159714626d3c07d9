// tree_attn_e4m3_f16.cu -- tree attention of fp16 queries over an e4m3 cache.
#include "tree_attn.cuh"

namespace relpos {
namespace tree {
cudaError_t run_e4m3_f16(const TreeParams& p, cudaStream_t s) { return run_format<__half, RELPOS_CACHE_E4M3>(p, s); }
}  // namespace tree
}  // namespace relpos
