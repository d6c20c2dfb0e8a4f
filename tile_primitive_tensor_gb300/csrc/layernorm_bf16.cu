// The layer norm's kernels for rows of bf16 (a file to a type, compiled side by side).
#include "layernorm_rows.cuh"

namespace tpg {
template cudaError_t layernorm_of<__nv_bfloat16>(const LayerNormOp&, cudaStream_t);
template cudaError_t layernorm_grad_of<__nv_bfloat16>(const LayerNormGradOp&, cudaStream_t);
}  // namespace tpg
