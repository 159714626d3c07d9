// tree_attn_int8_f16.cu -- tree attention of fp16 queries over an int8 cache.
#include "tree_attn.cuh"

namespace relpos {
namespace tree {
cudaError_t run_int8_f16(const TreeParams& p, cudaStream_t s) { return run_format<__half, RELPOS_CACHE_INT8>(p, s); }
}  // namespace tree
}  // namespace relpos
