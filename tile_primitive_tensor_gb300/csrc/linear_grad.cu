// Gradient of the linear layer's epilogue: dZ = dY act'(Z) in the operands'
// type, and the bias gradient sum_m dZ[m, n] from the unrounded 32-bit dZ.
//
// A block takes kCols columns and one strip of rows; its threads walk the strip
// with their columns' sums in registers, kRowLanes rows at a time, and the
// block's sums go to partial[strip]. A second launch adds the strips in order,
// so the result does not depend on the order in which blocks run. Bound by
// memory: dY and Z are read once and dZ written once.
#include "column_sum.cuh"
#include "elem.cuh"

namespace tpg {
namespace {

constexpr int kPer = 8;                  // columns of a thread
constexpr int kCols = 64 * kPer;         // columns of a block
constexpr int kRowLanes = 4;             // rows a block has in hand at a time

template <typename T, int ACT>
__device__ __forceinline__ void act_grad_strip(const ActGradOp& op, int strips, float (&sum)[kPer]) {
    const int t = threadIdx.x & 63, lane_row = threadIdx.x >> 6;
    const int64_t n0 = int64_t(blockIdx.x) * kCols + t;
    const int64_t m_begin = op.M * blockIdx.y / strips, m_end = op.M * (blockIdx.y + 1) / strips;
    const T* dY = static_cast<const T*>(op.dY);
    const T* Z = static_cast<const T*>(op.Z);
    T* dZ = static_cast<T*>(op.dZ);
    for (int64_t m = m_begin + lane_row; m < m_end; m += kRowLanes) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int64_t n = n0 + 64 * j;
            if (n >= op.N) continue;
            float d = to_f32(dY[m * op.lddy + n]);
            if constexpr (ACT != TPGEMM_ACT_NONE) {
                d *= act_bwd<ACT>(to_f32(Z[m * op.ldz + n]));
                // The two products read dZ in the operands' own type.
                if (dZ) dZ[m * op.lddz + n] = from_f32<T>(d);
            }
            sum[j] += d;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(64 * kRowLanes) act_grad_kernel(ActGradOp op, int strips) {
    __shared__ float s[kRowLanes][kCols];
    float sum[kPer] = {};
    with_act(op.act, [&](auto act) { act_grad_strip<T, decltype(act)::value>(op, strips, sum); });
    if (!op.partial) return;
    const int t = threadIdx.x & 63, lane_row = threadIdx.x >> 6;
#pragma unroll
    for (int j = 0; j < kPer; ++j) s[lane_row][t + 64 * j] = sum[j];
    __syncthreads();
    for (int c = threadIdx.x; c < kCols; c += 64 * kRowLanes) {
        const int64_t n = int64_t(blockIdx.x) * kCols + c;
        if (n >= op.N) continue;
        float v = 0.f;
#pragma unroll
        for (int r = 0; r < kRowLanes; ++r) v += s[r][c];
        op.partial[int64_t(blockIdx.y) * op.N + n] = v;
    }
}

}  // namespace

// Enough strips that the blocks fill the GPU about four times over, of at
// least 16 rows each.
int act_grad_strips(int64_t M, int64_t N) {
    const int64_t cb = (N + kCols - 1) / kCols;
    const int64_t want = cb > 0 ? (608 + cb - 1) / cb : 1;
    const int64_t most = (M + 15) / 16;
    return int(want < most ? want : (most < 1 ? 1 : most));
}

cudaError_t launch_act_grad(const ActGradOp& op, cudaStream_t stream) {
    const int strips = act_grad_strips(op.M, op.N);
    const int64_t cb = (op.N + kCols - 1) / kCols;
    if (cb > 0x7fffffff || strips > 65535) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(cb), static_cast<unsigned>(strips));
    if (op.dtype == TPGEMM_ELEM_F16)
        act_grad_kernel<__half><<<grid, 64 * kRowLanes, 0, stream>>>(op, strips);
    else
        act_grad_kernel<__nv_bfloat16><<<grid, 64 * kRowLanes, 0, stream>>>(op, strips);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !op.partial) return e;
    return launch_column_sum(op.partial, strips, op.N, op.dbias, op.grad, stream);
}

}  // namespace tpg
