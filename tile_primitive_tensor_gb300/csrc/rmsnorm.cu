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
//
// All of it is bound by memory. A row is read once into registers by a team of
// threads (a warp for narrow rows, else a block), eight neighbouring columns to
// a thread at a time so that each load moves 16 bytes, reduced, and written
// from the registers. Rows wider than a team's registers (16384 columns) are
// read twice, the second time from L2.
#include <algorithm>

#include "column_sum.cuh"
#include "launch.cuh"
#include "norm_rows.cuh"

namespace tpg {
namespace {

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

// Row scales take the maximum of |h gamma| along with the sum of squares, and
// rstd after it. Where 32 bits do not hold that maximum, the row's maximum is
// taken again, of |h rstd gamma|.
__device__ __forceinline__ bool off_scale(uint32_t amax) { return amax < 0x00800000u || amax >= 0x7f800000u; }

// A block's maximum within a few units of a power of two: its scale hangs on the
// roundings of rstd and of two products (one block in 10^6), so the power is
// compared with |h rstd gamma| to twice as many bits, rstd that of the 32-bit sum of
// squares. What that sum is off by (some 1e-7 of it) still decides one block in
// 2 x 10^7.
__device__ __forceinline__ bool near_power(uint32_t amax) {
    return ((amax + 8u) & 0x7fffffu) < 16u && amax >= 0x10000000u && amax < 0x70000000u;
}

// 1 / sqrt(sum / cols + eps) as a 32-bit value and what it is short of: one
// Newton step from the exact residual.
struct Rstd {
    float hi, lo;
};
__device__ __forceinline__ Rstd rstd_of(float sum, float cols, float eps) {
    const float q = sum / cols, ql = fmaf(-q, cols, sum) / cols;
    const float m = q + eps, t = m - q;
    const float ml = (q - (m - t)) + (eps - t) + ql;
    const float r = 1.f / sqrtf(m), rr = r * r;
    return {r, 0.5f * r * (fmaf(-m, rr, 1.f) - fmaf(m, fmaf(r, r, -rr), ml * rr))};
}
__device__ __forceinline__ bool reaches(float power, float h, const Rstd& r, float g) {
    const float p = h * r.hi, pl = fmaf(h, r.hi, -p) + h * r.lo;
    const float y = p * g, yl = fmaf(p, g, -y) + pl * g;
    return (fabsf(y) - power) + (y < 0.f ? -yl : yl) >= 0.f;
}

template <typename XT>
__device__ __forceinline__ float gamma_of(const RmsNormOp& op, int64_t c) {
    return op.g == TPGEMM_ELEM_F32 ? static_cast<const float*>(op.gamma)[c]
                                   : to_f32(static_cast<const XT*>(op.gamma)[c]);
}

// Stores one group of y (scaled for an 8-bit output) and, for MX, its scales.
// True: the group's block is near a power of two, see settle_block (elements
// that are not neighbours settle theirs here, before h is stored over X or R).
template <typename XT, bool VEC, int MODE>
__device__ __forceinline__ bool store_y(const RmsNormOp& op, int64_t row, const Cols<VEC>& c,
                                        float (&y)[8], float inv, float sum) {
    bool near = false;
    if constexpr (MODE == TPGEMM_SCALE_MX) {
        uint8_t* scale = static_cast<uint8_t*>(op.scale) + row * ((op.cols + 31) / 32);
        if constexpr (VEC) {  // four lanes hold 32 neighbouring columns
            uint32_t amax = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = max(amax, abs_bits(y[j]));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            near = near_power(amax);  // (the same in all four)
            const uint32_t code = mx_scale(amax, op.y, inv);
            if ((threadIdx.x & 3) == 0 && c.n > 0) scale[c.first / 32] = uint8_t(code);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] *= inv;
        } else {  // the warp holds 32 neighbouring columns of each j
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t amax = __reduce_max_sync(0xffffffffu, abs_bits(y[j]));
                if (near_power(amax)) {
                    const uint32_t power = (amax + 8u) & 0x7f800000u;
                    bool any = false;
                    if (j < c.n) {  // (h and gamma are read again, to hold no registers)
                        const int64_t at = c.first + int64_t(j) * c.step;
                        float h = to_f32(static_cast<const XT*>(op.X)[row * op.ldx + at]);
                        if (op.R) h += to_f32(static_cast<const XT*>(op.R)[row * op.ldr + at]);
                        any = reaches(__uint_as_float(power), h, rstd_of(sum, float(op.cols), op.eps),
                                      gamma_of<XT>(op, at));
                    }
                    amax = __any_sync(0xffffffffu, any) ? power : power - 1u;
                }
                const uint32_t code = mx_scale(amax, op.y, inv);
                if ((threadIdx.x & 31) == 0 && j < c.n)
                    scale[(c.first + int64_t(j) * c.step) / 32] = uint8_t(code);
                y[j] *= inv;
            }
        }
    } else if constexpr (MODE == TPGEMM_SCALE_ROW) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] *= inv;
    }
    const int64_t at = row * op.ldy;
    switch (op.y) {
        case TPGEMM_ELEM_F16: store_cols<__half, VEC>(op.Y, at, c, y); break;
        case TPGEMM_ELEM_BF16: store_cols<__nv_bfloat16, VEC>(op.Y, at, c, y); break;
        case TPGEMM_ELEM_E4M3: store_cols<e4m3, VEC>(op.Y, at, c, y); break;
        case TPGEMM_ELEM_E5M2: store_cols<e5m2, VEC>(op.Y, at, c, y); break;
        default: store_cols<float, VEC>(op.Y, at, c, y); break;
    }
    return near;
}

// Writes a block near a power of two again, by four lanes: the power in doubt is
// compared exactly. It comes after the row's stores, when registers are free
// (8192 x 8192 bf16: 88 us so, 89 without it, 110 in their midst).
template <typename XT>
__device__ __forceinline__ void settle_block(const RmsNormOp& op, int64_t row, const Cols<true>& c,
                                             const float (&h)[8], float sum) {
    const unsigned four = 0xfu << (threadIdx.x & 28);
    const Rstd rstd = rstd_of(sum, float(op.cols), op.eps);
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (c.n == 8) amax = max(amax, abs_bits(h[j] * rstd.hi * gamma_of<XT>(op, c.first + j)));
    amax = max(amax, __shfl_xor_sync(four, amax, 1));
    amax = max(amax, __shfl_xor_sync(four, amax, 2));
    const uint32_t power = (amax + 8u) & 0x7f800000u;
    bool any = false;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (c.n == 8) any = any || reaches(__uint_as_float(power), h[j], rstd, gamma_of<XT>(op, c.first + j));
    any = __any_sync(four, any);
    float inv;
    const uint32_t code = mx_scale(any ? power : power - 1u, op.y, inv);
    if (c.n != 8) return;
    if ((threadIdx.x & 3) == 0) static_cast<uint8_t*>(op.scale)[row * ((op.cols + 31) / 32) + c.first / 32] = uint8_t(code);
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = h[j] * rstd.hi * gamma_of<XT>(op, c.first + j) * inv;
    if (op.y == TPGEMM_ELEM_E4M3) store_cols<e4m3, true>(op.Y, row * op.ldy, c, y);
    else store_cols<e5m2, true>(op.Y, row * op.ldy, c, y);
}

// h of one group: x + r.
template <typename XT, bool VEC>
__device__ __forceinline__ void load_h(const RmsNormOp& op, int64_t row, const Cols<VEC>& c,
                                       float (&h)[8]) {
    load_cols<XT, VEC>(op.X, row * op.ldx, c, h);
    if (op.R) {
        float r[8];
        load_cols<XT, VEC>(op.R, row * op.ldr, c, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] += r[j];
    }
}

// What follows a row's loads: reduction, scale, and the stores of h and y.
template <typename XT, int V, bool VEC, bool WARP, int MODE>
__device__ __forceinline__ void finish_row(const RmsNormOp& op, int64_t row, int t, int team,
                                           const float (&h)[V][8], float2* s) {
    constexpr bool row_mode = MODE == TPGEMM_SCALE_ROW;
    float g[V][8];
    float ss = 0.f;
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        load_gamma<XT, VEC>(op.gamma, op.g, Cols<VEC>(i, t, team, op.cols), g[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            ss += h[i][j] * h[i][j];
            if constexpr (row_mode) amax = max(amax, abs_bits(h[i][j] * g[i][j]));
        }
    }
    team_sum_max<WARP>(ss, amax, s);
    const float rstd = 1.f / sqrtf(ss / float(op.cols) + op.eps);
    if (t == 0 && op.rstd) op.rstd[row] = rstd;
    float inv = 1.f;
    if constexpr (row_mode) {
        if (!off_scale(amax)) {
            amax = abs_bits(rstd * __uint_as_float(amax));
        } else {  // (the same for the whole team)
            amax = 0;
#pragma unroll
            for (int i = 0; i < V; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) amax = max(amax, abs_bits(h[i][j] * rstd * g[i][j]));
            team_max<WARP>(amax, s);
        }
        const float scale = row_scale(amax, op.y);
        if (t == 0) static_cast<float*>(op.scale)[row] = scale;
        inv = 1.f / scale;
    }
    uint32_t near = 0;  // groups whose block is near a power of two
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const Cols<VEC> c(i, t, team, op.cols);
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = h[i][j] * rstd * g[i][j];
        if (store_y<XT, VEC, MODE>(op, row, c, y, inv, ss)) near |= 1u << i;
        if (op.H) store_cols<XT, VEC>(op.H, row * op.ldh, c, h[i]);
    }
    if constexpr (MODE == TPGEMM_SCALE_MX && VEC) {
        if (near) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if ((near >> i) & 1u) settle_block<XT>(op, row, Cols<VEC>(i, t, team, op.cols), h[i], ss);
        }
    }
}

// Rows held in registers: V groups of eight columns to a thread; WARP: a row to
// a warp, else to a block. AHEAD: blocks stay and walk the rows grid-stride, and
// load the next row before the reduction of this one, which waits for all of
// it; else a team ends with its row and the blocks beside it keep memory busy.
template <typename XT, int V, bool VEC, bool WARP, int MODE, bool AHEAD = false>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : kMaxTeam) rmsnorm_kernel(const __grid_constant__ RmsNormOp op) {
    __shared__ float2 s[2][32];
    const int team = WARP ? 32 : int(blockDim.x);
    const int t = WARP ? int(threadIdx.x & 31) : int(threadIdx.x);
    int64_t row = WARP ? int64_t(blockIdx.x) * kWarpRows + (threadIdx.x >> 5) : int64_t(blockIdx.x);
    grid_launch_dependents();
    grid_dependency_wait();
    if (WARP && row >= op.rows) return;
    float h[V][8];
    if constexpr (!AHEAD) {
#pragma unroll
        for (int i = 0; i < V; ++i) load_h<XT, VEC>(op, row, Cols<VEC>(i, t, team, op.cols), h[i]);
        finish_row<XT, V, VEC, WARP, MODE>(op, row, t, team, h, s[0]);
    } else {
        Ahead<XT, VEC> x[V], r[V];
        auto fetch = [&](int64_t at) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const Cols<VEC> c(i, t, team, op.cols);
                x[i].load(op.X, at * op.ldx, c);
                if (op.R) r[i].load(op.R, at * op.ldr, c);
            }
        };
        fetch(row);
        for (int turn = 0; row < op.rows; row += gridDim.x, turn ^= 1) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                x[i].get(h[i]);
                if (op.R) {
                    float q[8];
                    r[i].get(q);
#pragma unroll
                    for (int j = 0; j < 8; ++j) h[i][j] += q[j];
                }
            }
            if (row + gridDim.x < op.rows) fetch(row + gridDim.x);
            finish_row<XT, V, VEC, WARP, MODE>(op, row, t, team, h, s[turn]);
        }
    }
}

// Rows of any width, a block to a row, read twice. Two blocks to an SM where 32
// registers do (2048 x 20480 bf16 with row scales 79 us, 112 with one).
template <typename XT, bool VEC, int MODE>
__global__ void __launch_bounds__(kMaxTeam, VEC && MODE != TPGEMM_SCALE_MX ? 2 : 1) rmsnorm_wide_kernel(const __grid_constant__ RmsNormOp op) {
    __shared__ float2 s[32];
    const int team = int(blockDim.x), t = int(threadIdx.x);
    const int64_t row = blockIdx.x;
    constexpr bool row_mode = MODE == TPGEMM_SCALE_ROW;
    const int64_t groups = (op.cols + 8 * team - 1) / (8 * team);
    float h[8], g[8];
    float ss = 0.f;
    uint32_t amax = 0;
    grid_launch_dependents();
    grid_dependency_wait();
    for (int64_t i = 0; i < groups; ++i) {
        const Cols<VEC> c(i, t, team, op.cols);
        load_h<XT, VEC>(op, row, c, h);
        if constexpr (row_mode) load_gamma<XT, VEC>(op.gamma, op.g, c, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            ss += h[j] * h[j];
            if constexpr (row_mode) amax = max(amax, abs_bits(h[j] * g[j]));
        }
    }
    team_sum_max<false>(ss, amax, s);
    const float rstd = 1.f / sqrtf(ss / float(op.cols) + op.eps);
    if (t == 0 && op.rstd) op.rstd[row] = rstd;
    float inv = 1.f;
    if constexpr (row_mode) {
        if (!off_scale(amax)) {
            amax = abs_bits(rstd * __uint_as_float(amax));
        } else {  // (the same for the whole block)
            amax = 0;
#pragma unroll 1
            for (int64_t i = 0; i < groups; ++i) {
                const Cols<VEC> c(i, t, team, op.cols);
                load_h<XT, VEC>(op, row, c, h);
                load_gamma<XT, VEC>(op.gamma, op.g, c, g);
#pragma unroll
                for (int j = 0; j < 8; ++j) amax = max(amax, abs_bits(h[j] * rstd * g[j]));
            }
            team_max<false>(amax, s);
        }
        const float scale = row_scale(amax, op.y);
        if (t == 0) static_cast<float*>(op.scale)[row] = scale;
        inv = 1.f / scale;
    }
    for (int64_t i = 0; i < groups; ++i) {
        const Cols<VEC> c(i, t, team, op.cols);
        load_h<XT, VEC>(op, row, c, h);
        load_gamma<XT, VEC>(op.gamma, op.g, c, g);
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = h[j] * rstd * g[j];
        const bool near = store_y<XT, VEC, MODE>(op, row, c, y, inv, ss);
        if constexpr (MODE == TPGEMM_SCALE_MX && VEC) {
            if (near) settle_block<XT>(op, row, c, h, ss);
        }
        if (op.H) store_cols<XT, VEC>(op.H, row * op.ldh, c, h);
    }
}

// ---------------------------------------------------------------- gradients
// Blocks walk the rows grid-stride, a team (a warp or the block) to a row, and
// keep the columns' sums of dgamma in registers; partial[block] gets the
// block's. A row's reduction is a wait for all of it, so the next row's loads
// are issued before it (without: 55 % of memory's rate at 8192 x 4096 bf16).
// Rows wider than a team's registers take the two kernels after this.
template <typename XT, int V, bool VEC, bool WARP, int MAXT = 512>
__global__ void __launch_bounds__(WARP ? 32 * kWarpRows : MAXT) rmsnorm_grad_kernel(const __grid_constant__ RmsNormGradOp op) {
    __shared__ float2 s[2][32];
    __shared__ float sum[WARP ? 8 * 32 * 8 * V : 1];
    // (Unpacked groups, or more threads, leave no registers for it.)
    constexpr bool kAhead = (VEC || V == 1) && (WARP || MAXT <= 512);
    const int team = WARP ? 32 : int(blockDim.x);
    const int t = WARP ? int(threadIdx.x & 31) : int(threadIdx.x);
    const int64_t teams = WARP ? kWarpRows : 1;
    const int64_t stride = int64_t(gridDim.x) * teams;
    grid_launch_dependents();
    grid_dependency_wait();
    float acc[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = 0.f;
    int64_t row = int64_t(blockIdx.x) * teams + (WARP ? threadIdx.x >> 5 : 0);
    Ahead<XT, VEC> a_dy[V], a_h[V], a_dh[V];
    float a_rstd = 0.f;
    auto fetch = [&](int64_t r) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const Cols<VEC> c(i, t, team, op.cols);
            a_dy[i].load(op.dY, r * op.lddy, c);
            a_h[i].load(op.H, r * op.ldh, c);
            if (op.dX && op.dH) a_dh[i].load(op.dH, r * op.lddh, c);
        }
        a_rstd = op.rstd[r];
    };
    if (kAhead && row < op.rows) fetch(row);
    for (int turn = 0; row < op.rows; row += stride, turn ^= 1) {
        if (!kAhead) fetch(row);
        float dy[V][8], n[V][8], d[V][8];
        const float rstd = a_rstd;
        float dot = 0.f;
        uint32_t unused = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            a_dy[i].get(dy[i]);
            a_h[i].get(n[i]);
            if (op.dX && op.dH) {
                a_dh[i].get(d[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) d[i][j] = 0.f;
            }
            float g[8];
            if (op.dX) load_gamma<XT, VEC>(op.gamma, op.g, Cols<VEC>(i, t, team, op.cols), g);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                n[i][j] *= rstd;
                acc[i][j] += dy[i][j] * n[i][j];
                if (op.dX) {
                    dy[i][j] *= g[j];
                    dot += dy[i][j] * n[i][j];
                }
            }
        }
        if (kAhead && row + stride < op.rows) fetch(row + stride);
        if (!op.dX) continue;
        team_sum_max<WARP>(dot, unused, s[turn]);
        dot /= float(op.cols);
#pragma unroll
        for (int i = 0; i < V; ++i) {
#pragma unroll
            for (int j = 0; j < 8; ++j) d[i][j] += rstd * (dy[i][j] - n[i][j] * dot);
            store_cols<XT, VEC>(op.dX, row * op.lddx, Cols<VEC>(i, t, team, op.cols), d[i]);
        }
    }
    if (!op.dgamma) return;
    float* out = op.partial + int64_t(blockIdx.x) * op.cols;
    if constexpr (WARP) {
        const int w = threadIdx.x >> 5;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[((w * V + i) * 8 + j) * 32 + t] = acc[i][j];
        __syncthreads();
        // The warps' sums in order; warp w finishes the groups w, w + 8, ...
        for (int k = w; k < V * 8; k += kWarpRows) {
            float v = 0.f;
#pragma unroll
            for (int r = 0; r < kWarpRows; ++r) v += sum[(r * V * 8 + k) * 32 + t];
            const Cols<VEC> c(k / 8, t, team, op.cols);
            if (k % 8 < c.n) out[c.first + int64_t(k % 8) * c.step] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) store_cols<float, VEC>(op.partial, int64_t(blockIdx.x) * op.cols,
                                                           Cols<VEC>(i, t, team, op.cols), acc[i]);
    }
}

template <typename XT>
__device__ __forceinline__ float gamma_at(const RmsNormGradOp& op, int64_t c) {
    return op.g == TPGEMM_ELEM_F32 ? static_cast<const float*>(op.gamma)[c]
                                   : to_f32(static_cast<const XT*>(op.gamma)[c]);
}

constexpr int kWideThreads = 512;

template <typename XT>
__global__ void __launch_bounds__(kWideThreads) rmsnorm_grad_wide_kernel(const RmsNormGradOp op) {
    __shared__ float2 s[32];
    const int64_t row = blockIdx.x;
    const XT* dy = static_cast<const XT*>(op.dY) + row * op.lddy;
    const XT* h = static_cast<const XT*>(op.H) + row * op.ldh;
    const float rstd = op.rstd[row];
    float dot = 0.f;
    uint32_t unused = 0;
    for (int64_t c = threadIdx.x; c < op.cols; c += kWideThreads)
        dot += to_f32(dy[c]) * gamma_at<XT>(op, c) * (to_f32(h[c]) * rstd);
    team_sum_max<false>(dot, unused, s);
    dot /= float(op.cols);
    for (int64_t c = threadIdx.x; c < op.cols; c += kWideThreads) {
        float d = rstd * (to_f32(dy[c]) * gamma_at<XT>(op, c) - to_f32(h[c]) * rstd * dot);
        if (op.dH) d += to_f32(static_cast<const XT*>(op.dH)[row * op.lddh + c]);
        static_cast<XT*>(op.dX)[row * op.lddx + c] = from_f32<XT>(d);
    }
}

// partial[strip][c] = sum over the strip's rows of dy h rstd.
template <typename XT>
__global__ void __launch_bounds__(256) rmsnorm_dgamma_kernel(const RmsNormGradOp op, int strips) {
    const int64_t c = int64_t(blockIdx.x) * 256 + threadIdx.x;
    const int64_t begin = op.rows * blockIdx.y / strips, end = op.rows * (blockIdx.y + 1) / strips;
    if (c >= op.cols) return;
    float v = 0.f;
    for (int64_t r = begin; r < end; ++r)
        v += to_f32(static_cast<const XT*>(op.dY)[r * op.lddy + c]) *
             (to_f32(static_cast<const XT*>(op.H)[r * op.ldh + c]) * op.rstd[r]);
    op.partial[int64_t(blockIdx.y) * op.cols + c] = v;
}

// Up to 512 columns a warp holds the row. Wider rows are a block's: for many
// rows two groups to a thread, which keeps more bytes on their way (8192 x 4096
// bf16 with residual: 44 us, 52 with one); for few rows, and for widths that are
// no multiple of eight, whose loads are narrow, one group, for the shortest time
// to the end of a row (4096 x 4100 bf16: 63 us, 62 with two; gradients 95, 133;
// 333 x 1001: 3.6, 4.8).
Spread spread_of(int64_t rows, int64_t cols) {
    const int64_t groups = (cols + 7) / 8;
    if (groups <= 64) return {32, groups <= 32 ? 1 : 2, true};
    if (cols > kMaxHeld) return {kMaxTeam, 0, false};
    const bool one = groups <= kMaxTeam && (rows <= 2 * kSms || cols % 8 != 0);
    const int64_t per = one ? groups : (groups + 1) / 2;
    return {int((per + 31) / 32 * 32), one ? 1 : 2, false};
}

template <typename XT, bool VEC, int MODE>
cudaError_t launch_norm(const RmsNormOp& op, cudaStream_t stream) {
    const Spread s = spread_of(op.rows, op.cols);
    if (s.v == 0) {
        if (op.rows > 0x7fffffff) return cudaErrorInvalidValue;
        return launch_dependent(rmsnorm_wide_kernel<XT, VEC, MODE>, dim3(unsigned(op.rows)),
                                dim3(unsigned(s.threads())), 0, stream, op);
    }
    int64_t blocks = (op.rows + s.rows() - 1) / s.rows();
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    auto fn = s.warp ? (s.v == 1 ? rmsnorm_kernel<XT, 1, VEC, true, MODE> : rmsnorm_kernel<XT, 2, VEC, true, MODE>)
              : s.v == 1 ? rmsnorm_kernel<XT, 1, VEC, false, MODE>
                         : rmsnorm_kernel<XT, 2, VEC, false, MODE>;
    if constexpr (VEC && (MODE == TPGEMM_SCALE_NONE || (MODE == TPGEMM_SCALE_MX && sizeof(XT) == 2))) {
        // Teams of 512 threads and more leave an SM two rows or one, too few to
        // hide each other's reductions: such rows are loaded ahead (bf16 with
        // residual, MX scales: 8192 x 8192 97 -> 88 us; no scales: 2048 x
        // 16384 55.9 -> 46.3 us; f32 8192 x 8192 179 -> 182, 98 -> 94 without
        // residual, 2048 x 16384 61 -> 55 so). Not with row scales, where it gains
        // nothing (bf16 90.5 either way, 2048 x 16384 55.3), nor f32 rows with MX
        // scales, which would spill (140 -> 186), nor narrower rows (8192 x 4096
        // 44.0 -> 46.4).
        if (s.v == 2 && s.team >= 512) {
            fn = rmsnorm_kernel<XT, 2, VEC, false, MODE, true>;
            blocks = std::min(blocks, int64_t(kSms) * (kMaxTeam / s.team));
        }
    }
    return launch_dependent(fn, dim3(unsigned(blocks)), dim3(unsigned(s.threads())), 0, stream, op);
}

template <typename XT>
cudaError_t launch_norm_typed(const RmsNormOp& op, cudaStream_t stream) {
    const bool vec = op.cols % 8 == 0 && rows_aligned(op.X, op.ldx, op.rows, op.x, 16) &&
                     rows_aligned(op.R, op.ldr, op.rows, op.x, 16) &&
                     rows_aligned(op.H, op.ldh, op.rows, op.x, 16) &&
                     rows_aligned(op.Y, op.ldy, op.rows, op.y, elem_size(op.y) == 1 ? 8 : 16) &&
                     rows_aligned(op.gamma, 0, 1, op.g, 16);
    const auto launch = [&](auto mode) {
        constexpr int kMode = decltype(mode)::value;
        return vec ? launch_norm<XT, true, kMode>(op, stream) : launch_norm<XT, false, kMode>(op, stream);
    };
    if (op.mode == TPGEMM_SCALE_MX) return launch(std::integral_constant<int, TPGEMM_SCALE_MX>());
    if (op.mode == TPGEMM_SCALE_ROW) return launch(std::integral_constant<int, TPGEMM_SCALE_ROW>());
    return launch(std::integral_constant<int, TPGEMM_SCALE_NONE>());
}

// Blocks of the register kernel: 512 threads to an SM, which is what its
// registers leave room for, and two rows to a team at the least, since each
// block's sums are written and read once more.
int grad_blocks(int64_t rows, const Spread& s) {
    const int64_t most = (rows + 2 * s.rows() - 1) / (2 * s.rows());
    const int64_t fill = kSms * (s.threads() >= 512 ? 1 : 512 / s.threads());
    return int(most < fill ? (most < 1 ? 1 : most) : fill);
}

int wide_strips(int64_t rows) {
    const int64_t most = (rows + 15) / 16;
    return int(most < 1 ? 1 : (most < 64 ? most : 64));
}

// (Teams of more than 512 threads have 64 registers to a thread: a variant of
// its own, so that the others are not held to that.)
template <typename XT, bool VEC>
void (*pick_grad(const Spread& s))(const RmsNormGradOp) {
    if (s.warp) return s.v == 1 ? rmsnorm_grad_kernel<XT, 1, VEC, true> : rmsnorm_grad_kernel<XT, 2, VEC, true>;
    if (s.team <= 512) return s.v == 1 ? rmsnorm_grad_kernel<XT, 1, VEC, false> : rmsnorm_grad_kernel<XT, 2, VEC, false>;
    return s.v == 1 ? rmsnorm_grad_kernel<XT, 1, VEC, false, kMaxTeam> : rmsnorm_grad_kernel<XT, 2, VEC, false, kMaxTeam>;
}

template <typename XT>
cudaError_t launch_grad_typed(const RmsNormGradOp& op, cudaStream_t stream) {
    const Spread s = spread_of(op.rows, op.cols);
    const int strips = rmsnorm_grad_strips(op.rows, op.cols);
    cudaError_t e = cudaSuccess;
    if (s.v == 0) {
        // dgamma first: dX may be written over dY or H.
        if (op.dgamma) {
            const dim3 grid(unsigned((op.cols + 255) / 256), static_cast<unsigned>(strips));
            rmsnorm_dgamma_kernel<XT><<<grid, 256, 0, stream>>>(op, strips);
            e = cudaGetLastError();
        }
        if (e == cudaSuccess && op.dX) {
            rmsnorm_grad_wide_kernel<XT><<<unsigned(op.rows), kWideThreads, 0, stream>>>(op);
            e = cudaGetLastError();
        }
    } else {
        const bool vec = op.cols % 8 == 0 && rows_aligned(op.dY, op.lddy, op.rows, op.x, 16) &&
                         rows_aligned(op.H, op.ldh, op.rows, op.x, 16) &&
                         rows_aligned(op.dH, op.lddh, op.rows, op.x, 16) &&
                         rows_aligned(op.dX, op.lddx, op.rows, op.x, 16) &&
                         rows_aligned(op.gamma, 0, 1, op.g, 16);
        const dim3 grid{unsigned(strips)}, block{unsigned(s.threads())};
        e = launch_dependent(vec ? pick_grad<XT, true>(s) : pick_grad<XT, false>(s), grid, block, 0,
                             stream, op);
    }
    if (e != cudaSuccess || !op.dgamma) return e;
    return launch_column_sum(op.partial, strips, op.cols, op.dgamma, op.grad, stream);
}

}  // namespace

cudaError_t launch_rmsnorm(const RmsNormOp& op, cudaStream_t stream) {
    if (op.x == TPGEMM_ELEM_F16) return launch_norm_typed<__half>(op, stream);
    if (op.x == TPGEMM_ELEM_BF16) return launch_norm_typed<__nv_bfloat16>(op, stream);
    return launch_norm_typed<float>(op, stream);
}

int rmsnorm_grad_strips(int64_t rows, int64_t cols) {
    const Spread s = spread_of(rows, cols);
    return s.v == 0 ? wide_strips(rows) : grad_blocks(rows, s);
}

cudaError_t launch_rmsnorm_grad(const RmsNormGradOp& op, cudaStream_t stream) {
    if (op.rows > 0x7fffffff) return cudaErrorInvalidValue;
    if (op.x == TPGEMM_ELEM_F16) return launch_grad_typed<__half>(op, stream);
    if (op.x == TPGEMM_ELEM_BF16) return launch_grad_typed<__nv_bfloat16>(op, stream);
    return launch_grad_typed<float>(op, stream);
}

}  // namespace tpg
