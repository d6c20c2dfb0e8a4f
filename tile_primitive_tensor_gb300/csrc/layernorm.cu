// Layer norm over rows, with dropout and the residual's addition before it and an
// optional 8-bit output with row scales; and its gradients.
//
//   h = r + drop(x),  mean and var of h's row,  rstd = 1 / sqrt(var + eps),
//   y = (h - mean) rstd gamma + beta,
//
// all in 32 bits from the sum x + r on; the stored h, y, mean and rstd are its
// roundings. var is the mean of (h - mean)^2, taken after the mean from the row
// in registers, so that it loses nothing to a large mean; what the 32-bit mean is
// off by comes out of the same pass, as the mean of h - mean, and is taken off.
// 8-bit rows: y / scale, scale = max(max|y| / top, 2^-126), as of the
// root-mean-square norm.
//
// Gradients, with n = (h - mean) rstd and w = dy gamma:
//   dt = rstd (w - mean(w) - n mean(w n)) + dh,  dr = dt,  dx = drop(dt),
//   dgamma = sum over rows of dy n,  dbeta = sum over rows of dy.
//
// Bound by memory: a row is read once, into the registers of a team of threads,
// eight neighbouring columns to a thread at a time. Rows wider than a team's
// registers (16384 columns) are read again from L2 for each pass.
#include <algorithm>

#include "column_sum.cuh"
#include "launch.cuh"
#include "norm_rows.cuh"
#include "philox.cuh"

namespace tpg {
namespace {

// Sums of a and b over a warp, or over the block through `s`. (Reductions that
// follow one another take different `s`; the one before last may be used again.)
template <bool WARP>
__device__ __forceinline__ void team_sum2(float& a, float& b, float2* s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if constexpr (!WARP) {
        const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) s[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        const float2 v = lane < nw ? s[lane] : make_float2(0.f, 0.f);
        a = v.x;
        b = v.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
    }
}

template <bool WARP>
__device__ __forceinline__ float team_sum1(float a, float2* s) {
    uint32_t unused = 0;
    team_sum_max<WARP>(a, unused, s);
    return a;
}

// Dropout of a thread's group; the whole warp calls it.
template <bool VEC>
__device__ __forceinline__ void drop_cols(const DropKey& k, int64_t row, const Cols<VEC>& c, float (&x)[8]) {
    if constexpr (VEC) {
        if (c.n == 8) {
            drop4(k, uint32_t(row), uint32_t(c.first / 4), x);
            drop4(k, uint32_t(row), uint32_t(c.first / 4 + 1), x + 4);
        }
    } else {
        drop8_apart(k, uint32_t(row), c.first, c.step, x);
    }
}

template <typename XT, bool VEC, bool DROP>
__device__ __forceinline__ void load_sum(const LayerNormOp& op, const DropKey& k, int64_t row, const Cols<VEC>& c,
                                         float (&h)[8]) {
    load_cols<XT, VEC>(op.X, row * op.ldx, c, h);
    if constexpr (DROP) drop_cols<VEC>(k, row, c, h);
    if (op.R) {
        float r[8];
        load_cols<XT, VEC>(op.R, row * op.ldr, c, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] += r[j];
    }
}

template <bool VEC>
__device__ __forceinline__ void store_y(const LayerNormOp& op, int64_t row, const Cols<VEC>& c, const float (&y)[8]) {
    const int64_t at = row * op.ldy;
    switch (op.y) {
        case TPGEMM_ELEM_F16: store_cols<__half, VEC>(op.Y, at, c, y); break;
        case TPGEMM_ELEM_BF16: store_cols<__nv_bfloat16, VEC>(op.Y, at, c, y); break;
        case TPGEMM_ELEM_E4M3: store_cols<e4m3, VEC>(op.Y, at, c, y); break;
        case TPGEMM_ELEM_E5M2: store_cols<e5m2, VEC>(op.Y, at, c, y); break;
        default: store_cols<float, VEC>(op.Y, at, c, y); break;
    }
}

// A row's mean as two 32-bit values (what the first is off by in the second),
// and rstd.
struct Stats {
    float mean, off, rstd;
};

// From the sums of h - mean and of its square.
__device__ __forceinline__ Stats stats_of(float mean, float d, float dd, float cols, float eps) {
    const float off = d / cols;
    float var = dd / cols - off * off;
    var = var < 0.f ? 0.f : var;  // (a NaN stays one)
    return {mean, off, 1.f / sqrtf(var + eps)};
}

// y of one group.
template <typename XT, bool VEC>
__device__ __forceinline__ void normalise(const LayerNormOp& op, const Stats& st, const Cols<VEC>& c,
                                          const float (&h)[8], float (&y)[8]) {
    float g[8], b[8];
    load_gamma<XT, VEC>(op.gamma, op.g, c, g);
    if (op.beta) {
        load_gamma<XT, VEC>(op.beta, op.g, c, b);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = fmaf((h[j] - st.mean - st.off) * st.rstd, g[j], b[j]);
}

// Rows held in registers: V groups of eight columns to a thread; WARP: a row to
// a warp, else to a block.
template <typename XT, int V, bool VEC, bool WARP, bool DROP>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : kMaxTeam)
    layernorm_kernel(const __grid_constant__ LayerNormOp op) {
    __shared__ float2 s[3][32];
    const int team = WARP ? 32 : int(blockDim.x);
    const int t = WARP ? int(threadIdx.x & 31) : int(threadIdx.x);
    const int64_t row = WARP ? int64_t(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : int64_t(blockIdx.x);
    grid_launch_dependents();
    grid_dependency_wait();
    if (WARP && row >= op.rows) return;
    DropKey k{};
    if constexpr (DROP) k = drop_key(op.drop);
    float h[V][8];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        load_sum<XT, VEC, DROP>(op, k, row, Cols<VEC>(i, t, team, op.cols), h[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += h[i][j];
    }
    const float mean = team_sum1<WARP>(sum, s[0]) / float(op.cols);
    float d = 0.f, dd = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const Cols<VEC> c(i, t, team, op.cols);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float e = j < c.n ? h[i][j] - mean : 0.f;
            d += e;
            dd += e * e;
        }
    }
    team_sum2<WARP>(d, dd, s[1]);
    const Stats st = stats_of(mean, d, dd, float(op.cols), op.eps);
    if (t == 0) {
        if (op.mean) op.mean[row] = st.mean + st.off;
        if (op.rstd) op.rstd[row] = st.rstd;
    }
    float inv = 1.f;
    if (op.mode == TPGEMM_SCALE_ROW) {
        float none = 0.f;
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const Cols<VEC> c(i, t, team, op.cols);
            float y[8];
            normalise<XT, VEC>(op, st, c, h[i], y);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < c.n) amax = max(amax, abs_bits(y[j]));
        }
        team_sum_max<WARP>(none, amax, s[2]);
        const float scale = row_scale(amax, op.y);
        if (t == 0) op.scale[row] = scale;
        inv = 1.f / scale;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const Cols<VEC> c(i, t, team, op.cols);
        float y[8];
        normalise<XT, VEC>(op, st, c, h[i], y);
        if (op.mode == TPGEMM_SCALE_ROW) {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] *= inv;
        }
        store_y<VEC>(op, row, c, y);
        if (op.H) store_cols<XT, VEC>(op.H, row * op.ldh, c, h[i]);
    }
}

// Rows of any width, a block to a row, read once for each pass.
template <typename XT, bool VEC, bool DROP>
__global__ void __launch_bounds__(kMaxTeam) layernorm_wide_kernel(const __grid_constant__ LayerNormOp op) {
    __shared__ float2 s[3][32];
    const int team = int(blockDim.x), t = int(threadIdx.x);
    const int64_t row = blockIdx.x;
    const int64_t groups = (op.cols + 8 * team - 1) / (8 * team);
    grid_launch_dependents();
    grid_dependency_wait();
    DropKey k{};
    if constexpr (DROP) k = drop_key(op.drop);
    float h[8], y[8];
    float sum = 0.f;
    for (int64_t i = 0; i < groups; ++i) {
        load_sum<XT, VEC, DROP>(op, k, row, Cols<VEC>(i, t, team, op.cols), h);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += h[j];
    }
    const float mean = team_sum1<false>(sum, s[0]) / float(op.cols);
    float d = 0.f, dd = 0.f;
    for (int64_t i = 0; i < groups; ++i) {
        const Cols<VEC> c(i, t, team, op.cols);
        load_sum<XT, VEC, DROP>(op, k, row, c, h);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float e = j < c.n ? h[j] - mean : 0.f;
            d += e;
            dd += e * e;
        }
    }
    team_sum2<false>(d, dd, s[1]);
    const Stats st = stats_of(mean, d, dd, float(op.cols), op.eps);
    if (t == 0) {
        if (op.mean) op.mean[row] = st.mean + st.off;
        if (op.rstd) op.rstd[row] = st.rstd;
    }
    float inv = 1.f;
    if (op.mode == TPGEMM_SCALE_ROW) {
        float none = 0.f;
        uint32_t amax = 0;
        for (int64_t i = 0; i < groups; ++i) {
            const Cols<VEC> c(i, t, team, op.cols);
            load_sum<XT, VEC, DROP>(op, k, row, c, h);
            normalise<XT, VEC>(op, st, c, h, y);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < c.n) amax = max(amax, abs_bits(y[j]));
        }
        team_sum_max<false>(none, amax, s[2]);
        const float scale = row_scale(amax, op.y);
        if (t == 0) op.scale[row] = scale;
        inv = 1.f / scale;
    }
    for (int64_t i = 0; i < groups; ++i) {
        const Cols<VEC> c(i, t, team, op.cols);
        load_sum<XT, VEC, DROP>(op, k, row, c, h);
        normalise<XT, VEC>(op, st, c, h, y);
        if (op.mode == TPGEMM_SCALE_ROW) {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] *= inv;
        }
        store_y<VEC>(op, row, c, y);
        if (op.H) store_cols<XT, VEC>(op.H, row * op.ldh, c, h);
    }
}

// ---------------------------------------------------------------- gradients
// Blocks walk the rows grid-stride, a team to a row, with the columns' sums of
// dgamma and dbeta in registers; partial[block] gets the block's, dgamma's
// columns and then dbeta's.
template <typename XT, int V, bool VEC, bool WARP, bool DROP>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : kMaxTeam)
    layernorm_grad_kernel(const __grid_constant__ LayerNormGradOp op) {
    __shared__ float2 s[2][32];
    __shared__ float sum[WARP ? 8 * 32 * 8 * V : 1];
    const int team = WARP ? 32 : int(blockDim.x);
    const int t = WARP ? int(threadIdx.x & 31) : int(threadIdx.x);
    const int64_t teams = WARP ? kWarpRows : 1;
    const int64_t stride = int64_t(gridDim.x) * teams;
    grid_launch_dependents();
    grid_dependency_wait();
    DropKey k{};
    if constexpr (DROP) k = drop_key(op.drop);
    const bool rows_wanted = op.dX || op.dR;
    float ag[V][8], ab[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) ag[i][j] = ab[i][j] = 0.f;
    int64_t row = int64_t(blockIdx.x) * teams + (WARP ? threadIdx.x >> 5 : 0);
    for (int turn = 0; row < op.rows; row += stride, turn ^= 1) {
        const float rstd = op.rstd[row], mean = op.mean[row];
        float w[V][8], n[V][8];
        float sw = 0.f, swn = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const Cols<VEC> c(i, t, team, op.cols);
            load_cols<XT, VEC>(op.dY, row * op.lddy, c, w[i]);
            load_cols<XT, VEC>(op.H, row * op.ldh, c, n[i]);
            float g[8];
            if (rows_wanted) load_gamma<XT, VEC>(op.gamma, op.g, c, g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                n[i][j] = (n[i][j] - mean) * rstd;
                ag[i][j] += w[i][j] * n[i][j];
                ab[i][j] += w[i][j];
                if (rows_wanted) {
                    w[i][j] *= g[j];  // (0 past the row)
                    sw += w[i][j];
                    swn += w[i][j] * n[i][j];
                }
            }
        }
        if (!rows_wanted) continue;
        team_sum2<WARP>(sw, swn, s[turn]);
        sw /= float(op.cols);
        swn /= float(op.cols);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const Cols<VEC> c(i, t, team, op.cols);
            float dt[8];
            if (op.dH) {
                load_cols<XT, VEC>(op.dH, row * op.lddh, c, dt);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) dt[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) dt[j] += rstd * (w[i][j] - sw - n[i][j] * swn);
            if (op.dR) store_cols<XT, VEC>(op.dR, row * op.lddr, c, dt);
            if (op.dX) {
                if constexpr (DROP) drop_cols<VEC>(k, row, c, dt);
                store_cols<XT, VEC>(op.dX, row * op.lddx, c, dt);
            }
        }
    }
    if (!op.partial) return;
    float* out = op.partial + int64_t(blockIdx.x) * 2 * op.cols;
    if constexpr (WARP) {
        const int w = threadIdx.x >> 5;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[((w * V + i) * 8 + j) * 32 + t] = which ? ab[i][j] : ag[i][j];
            __syncthreads();
            // The warps' sums in order; warp w finishes the groups w, w + 8, ...
            for (int q = w; q < V * 8; q += kWarpRows) {
                float v = 0.f;
#pragma unroll
                for (int r = 0; r < kWarpRows; ++r) v += sum[(r * V * 8 + q) * 32 + t];
                const Cols<VEC> c(q / 8, t, team, op.cols);
                if (q % 8 < c.n) out[which * op.cols + c.first + int64_t(q % 8) * c.step] = v;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const Cols<VEC> c(i, t, team, op.cols);
            store_cols<float, VEC>(out, 0, c, ag[i]);
            store_cols<float, VEC>(out, op.cols, c, ab[i]);
        }
    }
}

template <typename XT>
__device__ __forceinline__ float gamma_at(const LayerNormGradOp& op, int64_t c) {
    return op.g == TPGEMM_ELEM_F32 ? static_cast<const float*>(op.gamma)[c]
                                   : to_f32(static_cast<const XT*>(op.gamma)[c]);
}

// Rows wider than a team's registers: dt a row to a block, read twice, and the
// column sums apart.
template <typename XT, bool DROP>
__global__ void __launch_bounds__(kMaxTeam) layernorm_grad_wide_kernel(const __grid_constant__ LayerNormGradOp op) {
    __shared__ float2 s[32];
    const int64_t row = blockIdx.x;
    grid_launch_dependents();
    grid_dependency_wait();
    DropKey k{};
    if constexpr (DROP) k = drop_key(op.drop);
    const XT* dy = static_cast<const XT*>(op.dY) + row * op.lddy;
    const XT* h = static_cast<const XT*>(op.H) + row * op.ldh;
    const float rstd = op.rstd[row], mean = op.mean[row];
    float sw = 0.f, swn = 0.f;
    for (int64_t c = threadIdx.x; c < op.cols; c += kMaxTeam) {
        const float w = to_f32(dy[c]) * gamma_at<XT>(op, c);
        sw += w;
        swn += w * ((to_f32(h[c]) - mean) * rstd);
    }
    team_sum2<false>(sw, swn, s);
    sw /= float(op.cols);
    swn /= float(op.cols);
    for (int64_t c = threadIdx.x; c < op.cols; c += kMaxTeam) {
        float d = rstd * (to_f32(dy[c]) * gamma_at<XT>(op, c) - sw - (to_f32(h[c]) - mean) * rstd * swn);
        if (op.dH) d += to_f32(static_cast<const XT*>(op.dH)[row * op.lddh + c]);
        if (op.dR) static_cast<XT*>(op.dR)[row * op.lddr + c] = from_f32<XT>(d);
        if (op.dX) {
            if constexpr (DROP) {
                const uint4 w = philox(k, uint32_t(row), uint32_t(c / 4));
                const int q = int(c & 3);
                d = drop_one(k, q == 0 ? w.x : q == 1 ? w.y : q == 2 ? w.z : w.w, d);
            }
            static_cast<XT*>(op.dX)[row * op.lddx + c] = from_f32<XT>(d);
        }
    }
}

// partial[strip] = the strip's sums of dy n, then of dy.
template <typename XT>
__global__ void __launch_bounds__(256) layernorm_columns_kernel(const __grid_constant__ LayerNormGradOp op, int strips) {
    const int64_t c = int64_t(blockIdx.x) * 256 + threadIdx.x;
    const int64_t begin = op.rows * blockIdx.y / strips, end = op.rows * (blockIdx.y + 1) / strips;
    grid_launch_dependents();
    grid_dependency_wait();
    if (c >= op.cols) return;
    float g = 0.f, b = 0.f;
    for (int64_t r = begin; r < end; ++r) {
        const float dy = to_f32(static_cast<const XT*>(op.dY)[r * op.lddy + c]);
        g += dy * ((to_f32(static_cast<const XT*>(op.H)[r * op.ldh + c]) - op.mean[r]) * op.rstd[r]);
        b += dy;
    }
    float* out = op.partial + int64_t(blockIdx.y) * 2 * op.cols + c;
    out[0] = g;
    out[op.cols] = b;
}

// Up to 512 columns a warp holds the row; wider rows are a block's.
Spread spread_of(int64_t rows, int64_t cols) {
    const int64_t groups = (cols + 7) / 8;
    if (groups <= 64) return {32, groups <= 32 ? 1 : 2, true};
    if (cols > kMaxHeld) return {kMaxTeam, 0, false};
    const bool one = groups <= kMaxTeam && (rows <= 2 * kSms || cols % 8 != 0);
    const int64_t per = one ? groups : (groups + 1) / 2;
    return {int((per + 31) / 32 * 32), one ? 1 : 2, false};
}

template <typename XT, bool VEC, bool DROP>
cudaError_t launch_norm(const LayerNormOp& op, cudaStream_t stream) {
    const Spread s = spread_of(op.rows, op.cols);
    const int64_t blocks = s.v == 0 ? op.rows : (op.rows + s.rows() - 1) / s.rows();
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    auto fn = s.v == 0   ? layernorm_wide_kernel<XT, VEC, DROP>
              : s.warp   ? (s.v == 1 ? layernorm_kernel<XT, 1, VEC, true, DROP> : layernorm_kernel<XT, 2, VEC, true, DROP>)
              : s.v == 1 ? layernorm_kernel<XT, 1, VEC, false, DROP>
                         : layernorm_kernel<XT, 2, VEC, false, DROP>;
    return launch_dependent(fn, dim3(unsigned(blocks)), dim3(unsigned(s.threads())), 0, stream, op);
}

template <typename XT>
cudaError_t launch_norm_typed(const LayerNormOp& op, cudaStream_t stream) {
    const bool vec = op.cols % 8 == 0 && rows_aligned(op.X, op.ldx, op.rows, op.x, 16) &&
                     rows_aligned(op.R, op.ldr, op.rows, op.x, 16) &&
                     rows_aligned(op.H, op.ldh, op.rows, op.x, 16) &&
                     rows_aligned(op.Y, op.ldy, op.rows, op.y, elem_size(op.y) == 1 ? 8 : 16) &&
                     rows_aligned(op.gamma, 0, 1, op.g, 16) && rows_aligned(op.beta, 0, 1, op.g, 16);
    if (op.drop.on)
        return vec ? launch_norm<XT, true, true>(op, stream) : launch_norm<XT, false, true>(op, stream);
    return vec ? launch_norm<XT, true, false>(op, stream) : launch_norm<XT, false, false>(op, stream);
}

// Two rows to a team at the least, since each block's sums are written and read
// once more.
int grad_blocks(int64_t rows, const Spread& s) {
    const int64_t most = (rows + 2 * s.rows() - 1) / (2 * s.rows());
    const int64_t fill = kSms * (s.threads() >= 512 ? 1 : 512 / s.threads());
    return int(most < fill ? (most < 1 ? 1 : most) : fill);
}

int wide_strips(int64_t rows) {
    const int64_t most = (rows + 15) / 16;
    return int(most < 1 ? 1 : (most < 64 ? most : 64));
}

template <typename XT, bool VEC, bool DROP>
void (*pick_grad(const Spread& s))(const LayerNormGradOp) {
    if (s.warp)
        return s.v == 1 ? layernorm_grad_kernel<XT, 1, VEC, true, DROP> : layernorm_grad_kernel<XT, 2, VEC, true, DROP>;
    return s.v == 1 ? layernorm_grad_kernel<XT, 1, VEC, false, DROP> : layernorm_grad_kernel<XT, 2, VEC, false, DROP>;
}

template <typename XT>
cudaError_t launch_grad_typed(const LayerNormGradOp& op, cudaStream_t stream) {
    const Spread s = spread_of(op.rows, op.cols);
    const int strips = layernorm_grad_strips(op.rows, op.cols);
    const bool drop = op.drop.on != 0;
    cudaError_t e = cudaSuccess;
    if (s.v == 0) {
        // The columns first: dX or dR may be written over dY or H.
        if (op.partial) {
            const dim3 grid(unsigned((op.cols + 255) / 256), static_cast<unsigned>(strips));
            e = launch_dependent(layernorm_columns_kernel<XT>, grid, dim3(256), 0, stream, op, strips);
        }
        if (e == cudaSuccess && (op.dX || op.dR))
            e = launch_dependent(drop ? layernorm_grad_wide_kernel<XT, true> : layernorm_grad_wide_kernel<XT, false>,
                                 dim3(unsigned(op.rows)), dim3(kMaxTeam), 0, stream, op);
    } else {
        const bool vec = op.cols % 8 == 0 && rows_aligned(op.dY, op.lddy, op.rows, op.x, 16) &&
                         rows_aligned(op.H, op.ldh, op.rows, op.x, 16) &&
                         rows_aligned(op.dH, op.lddh, op.rows, op.x, 16) &&
                         rows_aligned(op.dX, op.lddx, op.rows, op.x, 16) &&
                         rows_aligned(op.dR, op.lddr, op.rows, op.x, 16) &&
                         rows_aligned(op.gamma, 0, 1, op.g, 16);
        auto fn = vec ? (drop ? pick_grad<XT, true, true>(s) : pick_grad<XT, true, false>(s))
                      : (drop ? pick_grad<XT, false, true>(s) : pick_grad<XT, false, false>(s));
        e = launch_dependent(fn, dim3(unsigned(strips)), dim3(unsigned(s.threads())), 0, stream, op);
    }
    if (e != cudaSuccess || !op.partial) return e;
    return launch_column_sums(op.partial, strips, op.cols, op.dgamma, op.dbeta, op.grad, stream);
}

}  // namespace

cudaError_t launch_layernorm(const LayerNormOp& op, cudaStream_t stream) {
    if (op.x == TPGEMM_ELEM_F16) return launch_norm_typed<__half>(op, stream);
    if (op.x == TPGEMM_ELEM_BF16) return launch_norm_typed<__nv_bfloat16>(op, stream);
    return launch_norm_typed<float>(op, stream);
}

int layernorm_grad_strips(int64_t rows, int64_t cols) {
    const Spread s = spread_of(rows, cols);
    return s.v == 0 ? wide_strips(rows) : grad_blocks(rows, s);
}

cudaError_t launch_layernorm_grad(const LayerNormGradOp& op, cudaStream_t stream) {
    if (op.rows > 0x7fffffff) return cudaErrorInvalidValue;
    if (op.x == TPGEMM_ELEM_F16) return launch_grad_typed<__half>(op, stream);
    if (op.x == TPGEMM_ELEM_BF16) return launch_grad_typed<__nv_bfloat16>(op, stream);
    return launch_grad_typed<float>(op, stream);
}

}  // namespace tpg
