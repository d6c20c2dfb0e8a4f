// Gradient of the linear layer's epilogue: dZ = dY act'(Z) in the operands'
// type, and the bias gradient sum_m dZ[m, n] from the unrounded 32-bit dZ; and
// the copy of an operand to rows that start on 16-byte boundaries.
//
// A block takes 512 columns and one strip of rows, a thread eight columns (16
// bytes of each matrix where rows allow it) of every fourth row; its threads
// walk the strip with their columns' sums in registers, and the block's sums
// go to partial[strip]. A second launch adds the strips in order, so the
// result does not depend on the order in which blocks run. Bound by memory:
// dY and Z are read once and dZ written once.
#include "column_sum.cuh"
#include "vec8.cuh"

namespace tpg {
namespace {

constexpr int kPer = 8;                  // columns of a thread
constexpr int kCols = 64 * kPer;         // columns of a block
constexpr int kRowLanes = 4;             // rows a block has in hand at a time

template <typename T, int ACT>
__device__ __forceinline__ void act_grad_strip(const ActGradOp& op, int strips, bool vec,
                                               float (&sum)[kPer]) {
    const int t = threadIdx.x & 63, lane_row = threadIdx.x >> 6;
    const int64_t n = int64_t(blockIdx.x) * kCols + kPer * t;
    const int64_t m_begin = op.M * blockIdx.y / strips, m_end = op.M * (blockIdx.y + 1) / strips;
    if (n >= op.N) return;
    const int cnt = op.N - n < kPer ? int(op.N - n) : kPer;
    vec = vec && cnt == kPer;
#pragma unroll 2
    for (int64_t m = m_begin + lane_row; m < m_end; m += kRowLanes) {
        float d[8];
        load8<T>(op.dY, m * op.lddy + n, vec, cnt, d);
        if constexpr (ACT != TPGEMM_ACT_NONE) {
            float z[8];
            load8<T>(op.Z, m * op.ldz + n, vec, cnt, z);
#pragma unroll
            for (int j = 0; j < 8; j += 2)
                split(mul(f2(d[j], d[j + 1]), act_bwd<ACT>(f2(z[j], z[j + 1]))), d[j], d[j + 1]);
            // The two products read dZ in the operands' own type.
            if (op.dZ) store8<T>(op.dZ, m * op.lddz + n, vec, cnt, d);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += d[j];
    }
}

template <typename T>
__global__ void __launch_bounds__(64 * kRowLanes)
    act_grad_kernel(const __grid_constant__ ActGradOp op, int strips, bool vec) {
    __shared__ float s[kRowLanes][kCols];
    grid_launch_dependents();
    grid_dependency_wait();
    float sum[kPer] = {};
    with_act(op.act, [&](auto act) {
        act_grad_strip<T, decltype(act)::value>(op, strips, vec, sum);
    });
    if (!op.partial) return;
    const int t = threadIdx.x & 63, lane_row = threadIdx.x >> 6;
#pragma unroll
    for (int j = 0; j < kPer; ++j) s[lane_row][j * 64 + t] = sum[j];
    __syncthreads();
    for (int c = threadIdx.x; c < kCols; c += 64 * kRowLanes) {
        const int64_t n = int64_t(blockIdx.x) * kCols + c;
        if (n >= op.N) continue;
        const int at = (c % kPer) * 64 + c / kPer;
        float v = 0.f;
#pragma unroll
        for (int r = 0; r < kRowLanes; ++r) v += s[r][at];
        op.partial[int64_t(blockIdx.y) * op.N + n] = v;
    }
}

// Rows of `bytes` bytes, `pitch` apart and anywhere in memory, to rows of whole
// 16-byte units; a thread to a unit. A unit with another one behind it in its
// row is read as five aligned words and shifted into place, the last one or
// two byte by byte.
__global__ void __launch_bounds__(256) align_rows_kernel(const uint8_t* src, int64_t rows, int64_t bytes,
                                                         int64_t pitch, uint8_t* dst, int64_t dst_pitch) {
    grid_launch_dependents();
    grid_dependency_wait();
    const int64_t u = int64_t(blockIdx.x) * 32 + (threadIdx.x & 31);
    if (16 * u >= bytes) return;
    for (int64_t r = int64_t(blockIdx.y) * 8 + (threadIdx.x >> 5); r < rows; r += int64_t(gridDim.y) * 8) {
        const uint8_t* p = src + r * pitch + 16 * u;
        uint32_t w[4] = {};
        if (16 * u + 32 <= bytes) {
            const uint32_t off = uint32_t(reinterpret_cast<uintptr_t>(p) & 3u);
            const uint32_t* q = reinterpret_cast<const uint32_t*>(p - off);
            uint32_t x[5];
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = q[i];
            x[4] = off ? q[4] : 0u;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(x[i], x[i + 1], 8 * off);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (16 * u + i < bytes) w[i / 4] |= uint32_t(p[i]) << (8 * (i % 4));
        }
        *reinterpret_cast<uint4*>(dst + r * dst_pitch + 16 * u) = make_uint4(w[0], w[1], w[2], w[3]);
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
    auto rows16 = [&](const void* p, int64_t ld) {
        return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (op.M <= 1 || ld % 8 == 0));
    };
    const bool vec = rows16(op.dY, op.lddy) && rows16(op.Z, op.ldz) && rows16(op.dZ, op.lddz);
    cudaError_t e = op.dtype == TPGEMM_ELEM_F16
                        ? launch_dependent(act_grad_kernel<__half>, grid, dim3(64 * kRowLanes), 0,
                                           stream, op, strips, vec)
                        : launch_dependent(act_grad_kernel<__nv_bfloat16>, grid, dim3(64 * kRowLanes), 0,
                                           stream, op, strips, vec);
    if (e != cudaSuccess || !op.partial) return e;
    return launch_column_sum(op.partial, strips, op.N, op.dbias, op.grad, stream);
}

cudaError_t launch_align_rows(const void* src, int64_t rows, int64_t bytes, int64_t pitch, void* dst,
                              int64_t dst_pitch, cudaStream_t stream) {
    const int64_t bx = (bytes + 511) / 512;
    int64_t by = (rows + 7) / 8;
    by = by < 1 ? 1 : (by > 4096 ? 4096 : by);
    if (bx > 0x7fffffff) return cudaErrorInvalidValue;
    return launch_dependent(align_rows_kernel, dim3(unsigned(bx), unsigned(by)), dim3(256), 0, stream,
                            static_cast<const uint8_t*>(src), rows, bytes, pitch,
                            static_cast<uint8_t*>(dst), dst_pitch);
}

}  // namespace tpg
