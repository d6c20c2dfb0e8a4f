// Root-mean-square norm over rows, with the residual's addition before it and
// an optional 8-bit output with scales after it; and its gradients.
//
//   h = x + r,  rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd gamma.
//
// h is summed, squared and normalised in 32 bits; the stored h, y and rstd are
// its roundings. 8-bit outputs are y / scale rounded to nearest even:
//   row scale:  scale = max(max|y| / top, 2^-126) per row (top: the type's
//               largest value), so an all-zero row divides by no zero;
//   MX scale:   2^e per 32 columns, e = floor(log2 max|y|) - emax of the type,
//               clamped to E8M0's range; values past the type's largest saturate.
// A row (block) that holds an infinity or a NaN gets a NaN scale, so that it
// reads back as NaN and not as a large finite value.
//
// Gradients, with n = h rstd and w = dy gamma:
//   dx = rstd (w - n mean(w n)) + dh,   dgamma = sum over rows of dy n.
#include "column_sum.cuh"
#include "elem.cuh"

namespace tpg {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float load_as(const void* p, int elem, int64_t i) {
    if (elem == TPGEMM_ELEM_F16) return to_f32(static_cast<const __half*>(p)[i]);
    if (elem == TPGEMM_ELEM_BF16) return to_f32(static_cast<const __nv_bfloat16*>(p)[i]);
    return static_cast<const float*>(p)[i];
}

__device__ __forceinline__ void store_as(void* p, int elem, int64_t i, float v) {
    switch (elem) {
        case TPGEMM_ELEM_F16: static_cast<__half*>(p)[i] = from_f32<__half>(v); break;
        case TPGEMM_ELEM_BF16: static_cast<__nv_bfloat16*>(p)[i] = from_f32<__nv_bfloat16>(v); break;
        case TPGEMM_ELEM_E4M3: static_cast<e4m3*>(p)[i] = from_f32<e4m3>(v); break;
        case TPGEMM_ELEM_E5M2: static_cast<e5m2*>(p)[i] = from_f32<e5m2>(v); break;
        default: static_cast<float*>(p)[i] = v; break;
    }
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Largest |value| of a set as the 32-bit pattern: an integer maximum, so that
// infinities and NaN (the largest patterns) are kept.
__device__ __forceinline__ float row_scale(uint32_t amax, int elem) {
    const float top = elem == TPGEMM_ELEM_E4M3 ? 448.f : 57344.f;
    if (amax >= 0x7f800000u) return __uint_as_float(0x7fffffffu);
    return fmaxf(__uint_as_float(amax) / top, 1.17549435e-38f);
}

// E8M0 code of a block with the given largest |value|, and 1 / its scale.
__device__ __forceinline__ uint32_t mx_scale(uint32_t amax, int elem, float& inv) {
    if (amax >= 0x7f800000u) {
        inv = __uint_as_float(0x7fffffffu);
        return 255u;
    }
    const int e = max(int(amax >> 23) - 127 - (elem == TPGEMM_ELEM_E4M3 ? 8 : 15), -127);
    inv = __uint_as_float(uint32_t(127 - e) << 23);
    return uint32_t(e + 127);
}

// Sum of a and maximum of b over the block, in every thread.
__device__ __forceinline__ void block_sum_max(float& a, uint32_t& b) {
    __shared__ float sa[32];
    __shared__ uint32_t sb[32];
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    b = __reduce_max_sync(0xffffffffu, b);
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
    __syncthreads();
    if (lane == 0) {
        sa[w] = a;
        sb[w] = b;
    }
    __syncthreads();
    a = 0.f;
    b = 0u;
    for (int i = 0; i < nw; ++i) {
        a += sa[i];
        b = max(b, sb[i]);
    }
}

// One row per block, any width: a first pass over the row for its sum of
// squares (and largest |h gamma|), a second that reads it again and writes.
__global__ void __launch_bounds__(kThreads) rmsnorm_wide_kernel(RmsNormOp op) {
    const int64_t row = blockIdx.x;
    const int64_t xo = row * op.ldx, ro = row * op.ldr, ho = row * op.ldh, yo = row * op.ldy;
    auto h_at = [&](int64_t c) {
        float h = load_as(op.X, op.x, xo + c);
        if (op.R) h += load_as(op.R, op.x, ro + c);
        return h;
    };
    float ss = 0.f;
    uint32_t amax = 0;
    for (int64_t c = threadIdx.x; c < op.cols; c += kThreads) {
        const float h = h_at(c);
        ss += h * h;
        if (op.mode == TPGEMM_SCALE_ROW) amax = max(amax, abs_bits(h * load_as(op.gamma, op.g, c)));
    }
    block_sum_max(ss, amax);
    const float rstd = 1.f / sqrtf(ss / float(op.cols) + op.eps);
    if (threadIdx.x == 0 && op.rstd) op.rstd[row] = rstd;
    float inv = 1.f;
    if (op.mode == TPGEMM_SCALE_ROW) {
        const float scale = row_scale(abs_bits(rstd * __uint_as_float(amax)), op.y);
        if (threadIdx.x == 0) static_cast<float*>(op.scale)[row] = scale;
        inv = 1.f / scale;
    }
    const int64_t blocks = (op.cols + 31) / 32;
    for (int64_t c0 = 0; c0 < op.cols; c0 += kThreads) {
        const int64_t c = c0 + threadIdx.x;
        float y = 0.f;
        if (c < op.cols) {
            const float h = h_at(c);
            if (op.H) store_as(op.H, op.x, ho + c, h);
            y = h * rstd * load_as(op.gamma, op.g, c);
        }
        if (op.mode == TPGEMM_SCALE_MX) {  // a warp holds one block of 32 columns
            const uint32_t code = mx_scale(__reduce_max_sync(0xffffffffu, abs_bits(y)), op.y, inv);
            if ((threadIdx.x & 31) == 0 && c < op.cols)
                static_cast<uint8_t*>(op.scale)[row * blocks + c / 32] = uint8_t(code);
        }
        if (c < op.cols) store_as(op.Y, op.y, yo + c, op.mode == TPGEMM_SCALE_NONE ? y : y * inv);
    }
}

__global__ void __launch_bounds__(kThreads) rmsnorm_grad_wide_kernel(RmsNormGradOp op) {
    const int64_t row = blockIdx.x;
    const int64_t yo = row * op.lddy, ho = row * op.ldh, do_ = row * op.lddh, xo = row * op.lddx;
    const float rstd = op.rstd[row];
    float dot = 0.f;
    uint32_t unused = 0;
    for (int64_t c = threadIdx.x; c < op.cols; c += kThreads)
        dot += load_as(op.dY, op.x, yo + c) * load_as(op.gamma, op.g, c) *
               (load_as(op.H, op.x, ho + c) * rstd);
    block_sum_max(dot, unused);
    dot /= float(op.cols);
    for (int64_t c = threadIdx.x; c < op.cols; c += kThreads) {
        const float n = load_as(op.H, op.x, ho + c) * rstd;
        float d = rstd * (load_as(op.dY, op.x, yo + c) * load_as(op.gamma, op.g, c) - n * dot);
        if (op.dH) d += load_as(op.dH, op.x, do_ + c);
        store_as(op.dX, op.x, xo + c, d);
    }
}

// partial[strip][c] = sum over the strip's rows of dy h rstd.
__global__ void __launch_bounds__(kThreads) rmsnorm_dgamma_kernel(RmsNormGradOp op, int strips) {
    const int64_t c = int64_t(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t begin = op.rows * blockIdx.y / strips, end = op.rows * (blockIdx.y + 1) / strips;
    if (c >= op.cols) return;
    float v = 0.f;
    for (int64_t r = begin; r < end; ++r)
        v += load_as(op.dY, op.x, r * op.lddy + c) * (load_as(op.H, op.x, r * op.ldh + c) * op.rstd[r]);
    op.partial[int64_t(blockIdx.y) * op.cols + c] = v;
}

}  // namespace

cudaError_t launch_rmsnorm(const RmsNormOp& op, cudaStream_t stream) {
    if (op.rows > 0x7fffffff) return cudaErrorInvalidValue;
    rmsnorm_wide_kernel<<<unsigned(op.rows), kThreads, 0, stream>>>(op);
    return cudaGetLastError();
}

int rmsnorm_grad_strips(int64_t rows, int64_t cols) {
    const int64_t most = (rows + 15) / 16;
    return int(most < 1 ? 1 : (most < 152 ? most : 152));
}

cudaError_t launch_rmsnorm_grad(const RmsNormGradOp& op, cudaStream_t stream) {
    if (op.rows > 0x7fffffff) return cudaErrorInvalidValue;
    // dgamma first: dX may be written over dY or H.
    if (op.dgamma) {
        const int strips = rmsnorm_grad_strips(op.rows, op.cols);
        const dim3 grid(unsigned((op.cols + kThreads - 1) / kThreads), static_cast<unsigned>(strips));
        rmsnorm_dgamma_kernel<<<grid, kThreads, 0, stream>>>(op, strips);
        cudaError_t e = cudaGetLastError();
        if (e == cudaSuccess)
            e = launch_column_sum(op.partial, strips, op.cols, op.dgamma, op.grad, stream);
        if (e != cudaSuccess) return e;
    }
    if (op.dX && op.rows > 0) rmsnorm_grad_wide_kernel<<<unsigned(op.rows), kThreads, 0, stream>>>(op);
    return cudaGetLastError();
}

}  // namespace tpg
