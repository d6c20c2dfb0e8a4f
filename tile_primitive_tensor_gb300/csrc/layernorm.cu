// The layer norm's launches, by the type of the rows.
#include "layernorm_rows.cuh"

namespace tpg {

extern template cudaError_t layernorm_of<__half>(const LayerNormOp&, cudaStream_t);
extern template cudaError_t layernorm_of<__nv_bfloat16>(const LayerNormOp&, cudaStream_t);
extern template cudaError_t layernorm_of<float>(const LayerNormOp&, cudaStream_t);
extern template cudaError_t layernorm_grad_of<__half>(const LayerNormGradOp&, cudaStream_t);
extern template cudaError_t layernorm_grad_of<__nv_bfloat16>(const LayerNormGradOp&, cudaStream_t);
extern template cudaError_t layernorm_grad_of<float>(const LayerNormGradOp&, cudaStream_t);

cudaError_t launch_layernorm(const LayerNormOp& op, cudaStream_t stream) {
    if (op.x == TPGEMM_ELEM_F16) return layernorm_of<__half>(op, stream);
    if (op.x == TPGEMM_ELEM_BF16) return layernorm_of<__nv_bfloat16>(op, stream);
    return layernorm_of<float>(op, stream);
}

int layernorm_grad_strips(int64_t rows, int64_t cols) {
    if (cols > kMaxHeld) return wide_strips(rows);
    // (The workspace does not hang on the rows' type and place.)
    int most = 1;
    for (const int elem : {TPGEMM_ELEM_F16, TPGEMM_ELEM_F32})
        for (const bool aligned : {false, true})
            most = std::max(most, grad_row_blocks(rows, row_spread(rows, cols, elem, true, aligned)));
    return most;
}

cudaError_t launch_layernorm_grad(const LayerNormGradOp& op, cudaStream_t stream) {
    if (op.rows > 0x7fffffff) return cudaErrorInvalidValue;
    if (op.x == TPGEMM_ELEM_F16) return layernorm_grad_of<__half>(op, stream);
    if (op.x == TPGEMM_ELEM_BF16) return layernorm_grad_of<__nv_bfloat16>(op, stream);
    return layernorm_grad_of<float>(op, stream);
}

}  // namespace tpg
