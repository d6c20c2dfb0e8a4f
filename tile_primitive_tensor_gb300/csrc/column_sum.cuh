// out[n] = sum over strips s of partial[s][n], always in the same order, rounded
// once; or the same with two outputs side by side in `partial`.
#pragma once

#include "elem.cuh"
#include "launch.cuh"
#include "ptx.cuh"

namespace tpg {
namespace {

// 32 columns to a block, its 32 warps taking every 32nd strip.
// Columns from `first` on are out2's. Either output may be null.
template <typename O>
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* partial, int strips, int64_t cols, O* out,
                                                          int64_t first, O* out2) {
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
    O* const to = c < first ? out : out2;
    if (lane == 0 && c < cols && to) to[c < first ? c : c - first] = from_f32<O>(v);
}

template <typename O>
cudaError_t launch_column_sum_typed(const float* partial, int strips, int64_t cols, void* out, int64_t first,
                                    void* out2, cudaStream_t stream) {
    const int64_t blocks = (cols + 31) / 32;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_dependent(column_sum_kernel<O>, dim3(unsigned(blocks)), dim3(1024), 0, stream, partial, strips,
                            cols, static_cast<O*>(out), first, static_cast<O*>(out2));
}

// partial[strip] holds out's `cols` sums and then out2's.
inline cudaError_t launch_column_sums(const float* partial, int strips, int64_t cols, void* out, void* out2,
                                      int elem, cudaStream_t stream) {
    auto fn = elem == TPGEMM_ELEM_F16    ? launch_column_sum_typed<__half>
              : elem == TPGEMM_ELEM_BF16 ? launch_column_sum_typed<__nv_bfloat16>
                                         : launch_column_sum_typed<float>;
    return fn(partial, strips, 2 * cols, out, cols, out2, stream);
}

inline cudaError_t launch_column_sum(const float* partial, int strips, int64_t cols, void* out, int elem,
                                     cudaStream_t stream) {
    auto fn = elem == TPGEMM_ELEM_F16    ? launch_column_sum_typed<__half>
              : elem == TPGEMM_ELEM_BF16 ? launch_column_sum_typed<__nv_bfloat16>
                                         : launch_column_sum_typed<float>;
    return fn(partial, strips, cols, out, cols, nullptr, stream);
}

}  // namespace
}  // namespace tpg
