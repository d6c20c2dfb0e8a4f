// out[n] = sum over strips s of partial[s][n], always in the same order, rounded
// once.
#pragma once

#include "elem.cuh"
#include "launch.cuh"
#include "ptx.cuh"

namespace tpg {
namespace {

// 32 columns to a block, its 32 warps taking every 32nd strip.
template <typename O>
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* partial, int strips,
                                                          int64_t cols, O* out) {
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t n = int64_t(blockIdx.x) * 32 + lane;
    grid_launch_dependents();
    grid_dependency_wait();
    float v = 0.f;
    if (n < cols)
#pragma unroll 4
        for (int i = w; i < strips; i += 32) v += partial[int64_t(i) * cols + n];
    s[w][lane] = v;
    __syncthreads();
    // Warp w adds column w's sums.
    v = s[lane][w];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int64_t c = int64_t(blockIdx.x) * 32 + w;
    if (lane == 0 && c < cols) out[c] = from_f32<O>(v);
}

inline cudaError_t launch_column_sum(const float* partial, int strips, int64_t cols, void* out,
                                     int elem, cudaStream_t stream) {
    const int64_t blocks = (cols + 31) / 32;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    const dim3 g{unsigned(blocks)}, b{1024};
    if (elem == TPGEMM_ELEM_F16)
        return launch_dependent(column_sum_kernel<__half>, g, b, 0, stream, partial, strips, cols,
                                static_cast<__half*>(out));
    if (elem == TPGEMM_ELEM_BF16)
        return launch_dependent(column_sum_kernel<__nv_bfloat16>, g, b, 0, stream, partial, strips, cols,
                                static_cast<__nv_bfloat16*>(out));
    return launch_dependent(column_sum_kernel<float>, g, b, 0, stream, partial, strips, cols,
                            static_cast<float*>(out));
}

}  // namespace
}  // namespace tpg
