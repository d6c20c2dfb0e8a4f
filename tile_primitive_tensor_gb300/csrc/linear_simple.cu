// The linear layer's product in its simplest form, for every type, layout and
// size: a 64 x 64 tile of the output per block, 32-bit multiply-adds, operands
// read one element at a time through their strides. Bound by the 32-bit FMA
// rate and its scalar loads.
#include "elem.cuh"

namespace tpg {
namespace {

constexpr int kT = 64, kTK = 16;

template <typename T>
__device__ __forceinline__ float load_elem(const Operand& o, int64_t r, int64_t k) {
    return to_f32(static_cast<const T*>(o.p)[o.mn ? k * o.ld + r : r * o.ld + k]);
}

template <typename T, typename O>
__global__ void __launch_bounds__(256) linear_simple_kernel(LinearOp op) {
    __shared__ float sa[kTK][kT + 1], sb[kTK][kT + 1];
    const int64_t tiles_n = (op.N + kT - 1) / kT;
    const int64_t m0 = (blockIdx.x / tiles_n) * kT, n0 = (blockIdx.x % tiles_n) * kT;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < op.K; k0 += kTK) {
        for (int i = threadIdx.x; i < kT * kTK; i += 256) {
            // Consecutive threads along the operand's contiguous axis.
            const int ra = op.a.mn ? i % kT : i / kTK, ka = op.a.mn ? i / kT : i % kTK;
            const int rb = op.b.mn ? i % kT : i / kTK, kb = op.b.mn ? i / kT : i % kTK;
            sa[ka][ra] = (m0 + ra < op.M && k0 + ka < op.K) ? load_elem<T>(op.a, m0 + ra, k0 + ka) : 0.f;
            sb[kb][rb] = (n0 + rb < op.N && k0 + kb < op.K) ? load_elem<T>(op.b, n0 + rb, k0 + kb) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kTK; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] += sa[k][ty + 16 * i] * sb[k][tx + 16 * j];
        __syncthreads();
    }
    with_act(op.e.act, [&](auto act) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
                if (m < op.M && n < op.N)
                    epilogue_one<O, decltype(act)::value>(op.e, m, n, acc[i][j]);
            }
    });
}

template <typename T>
cudaError_t launch_typed(const LinearOp& op, cudaStream_t stream) {
    const int64_t tiles = ((op.N + kT - 1) / kT) * ((op.M + kT - 1) / kT);
    if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
    const unsigned grid = unsigned(tiles);
    if (op.e.out == TPGEMM_ELEM_F16)
        linear_simple_kernel<T, __half><<<grid, 256, 0, stream>>>(op);
    else if (op.e.out == TPGEMM_ELEM_BF16)
        linear_simple_kernel<T, __nv_bfloat16><<<grid, 256, 0, stream>>>(op);
    else
        linear_simple_kernel<T, float><<<grid, 256, 0, stream>>>(op);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_simple(const LinearOp& op, cudaStream_t stream) {
    switch (op.dtype) {
        case TPGEMM_ELEM_F16: return launch_typed<__half>(op, stream);
        case TPGEMM_ELEM_BF16: return launch_typed<__nv_bfloat16>(op, stream);
        case TPGEMM_ELEM_E4M3: return launch_typed<e4m3>(op, stream);
        default: return launch_typed<e5m2>(op, stream);
    }
}

}  // namespace tpg
