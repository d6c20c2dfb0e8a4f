// Dropout: Y = R + X / (1 - p) where the element's random word says so, R
// elsewhere (philox.cuh). Its gradient is the same with dY for X and no R.
//
// A thread takes eight neighbouring columns, 16 bytes of each matrix of 16-bit
// elements, and walks the matrix grid-stride. Rows that do not start on 16-byte
// boundaries, or widths that are no multiple of eight, move element by element.
// 8192 x 8192 bf16 with residual 65 us (93 % of memory's rate), without 62 (65 %): there
// the words' products keep their pipe busy for 70 % of the time and a third of the warps'
// waiting is for loads, which a thread asks for after the words of the group before; the
// two add up in part. 8192 x 4099 79 us (aligned 16 bytes joined and turned: 84). Two groups
// of columns to a thread at a time gained nothing (79 us at 8192 x 8192), nor did four
// of one row (78): warps, which have the registers then, are what hides memory here.
#include <algorithm>

#include "launch.cuh"
#include "norm_rows.cuh"
#include "philox.cuh"

namespace tpg {
namespace {

constexpr int kDropThreads = 256;
constexpr int kPer = 8;  // columns of a thread

// Groups of kPer columns from the thread's first on; step_rows, step_groups: the
// grid's number of threads as whole rows and a rest.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(const __grid_constant__ DropoutOp op, int64_t groups,
                                                               int64_t step_rows, int64_t step_groups) {
    const uint64_t at = uint64_t(blockIdx.x) * kDropThreads + threadIdx.x;
    int64_t row = int64_t(at / uint64_t(groups)), g = int64_t(at % uint64_t(groups));
    grid_launch_dependents();
    grid_dependency_wait();
    const DropOffset offset = drop_offset(op.drop);
    const float scale = op.drop.on ? op.drop.scale : 1.f;
    for (; row < op.rows; row += step_rows, g += step_groups) {
        if (g >= groups) {
            g -= groups;
            if (++row >= op.rows) break;
        }
        const int64_t c = g * kPer;
        const int n = VEC ? kPer : int(min(int64_t(kPer), op.cols - c));
        float x[8], r[8];
        load8<T>(op.X, row * op.ldx + c, VEC, n, x);
        if (op.R) load8<T>(op.R, row * op.ldr + c, VEC, n, r);
        if (op.drop.on) {
            const DropRow w = drop_row(op.drop, offset, uint32_t(row));
            keep4(op.drop, w, uint32_t(2 * g), x);
            keep4(op.drop, w, uint32_t(2 * g + 1), x + 4);
        }
        if (op.R) {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = fmaf(x[j], scale, r[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] *= scale;
        }
        store8<T>(op.Y, row * op.ldy + c, VEC, n, x);
    }
}

template <typename T>
cudaError_t launch_dropout_typed(const DropoutOp& op, cudaStream_t stream) {
    const bool vec = op.cols % kPer == 0 && rows_aligned(op.X, op.ldx, op.rows, op.elem, 16) &&
                     rows_aligned(op.R, op.ldr, op.rows, op.elem, 16) &&
                     rows_aligned(op.Y, op.ldy, op.rows, op.elem, 16);
    const int64_t groups = (op.cols + kPer - 1) / kPer;
    const int64_t want = (op.rows * groups + kDropThreads - 1) / kDropThreads;
    const int64_t blocks = std::min<int64_t>(want, 8 * kSms);
    const int64_t threads = blocks * kDropThreads;
    return launch_dependent(vec ? dropout_kernel<T, true> : dropout_kernel<T, false>, dim3(unsigned(blocks)),
                            dim3(kDropThreads), 0, stream, op, groups, threads / groups, threads % groups);
}

}  // namespace

cudaError_t launch_dropout(const DropoutOp& op, cudaStream_t stream) {
    if (op.elem == TPGEMM_ELEM_F16) return launch_dropout_typed<__half>(op, stream);
    if (op.elem == TPGEMM_ELEM_BF16) return launch_dropout_typed<__nv_bfloat16>(op, stream);
    return launch_dropout_typed<float>(op, stream);
}

}  // namespace tpg
