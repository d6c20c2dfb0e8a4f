// The layer norm's kernels for rows of f32 (a file to a type, compiled side by side).
#include "layernorm_rows.cuh"

namespace tpg {
template cudaError_t layernorm_of<float>(const LayerNormOp&, cudaStream_t);
template cudaError_t layernorm_grad_of<float>(const LayerNormGradOp&, cudaStream_t);
}  // namespace tpg
