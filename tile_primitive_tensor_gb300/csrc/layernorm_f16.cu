// The layer norm's kernels for rows of f16 (a file to a type, compiled side by side).
#include "layernorm_rows.cuh"

namespace tpg {
template cudaError_t layernorm_of<__half>(const LayerNormOp&, cudaStream_t);
template cudaError_t layernorm_grad_of<__half>(const LayerNormGradOp&, cudaStream_t);
}  // namespace tpg
