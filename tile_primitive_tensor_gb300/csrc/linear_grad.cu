// Gradient of the linear layer's epilogue: dZ = dY act'(Z) in the operands'
// type, and the bias gradient sum_m dZ[m, n] from the unrounded 32-bit dZ; and
// the copy of an operand to rows that start on 16-byte boundaries.
//
// A thread takes eight columns (16 bytes of each matrix where rows allow it) of
// every 4th row of a block's strip, with their sums in registers; a block takes
// 512 columns and its sums go to partial[strip]. A second launch adds the
// strips in order, so the result does not depend on the order in which blocks
// run. Few rows are one strip, of blocks of 64 columns and 32 rows at a time,
// and end in dbias itself. dY and Z are read once and dZ is written once; with
// an activation the bound is between memory and the instructions of its
// derivative (about 24 an element): dbias of 8192 x 8192 bf16 34 us without one
// (58 % of memory's rate), 60 with silu, 64 with gelu, 67 with gelu_tanh. 64
// registers, so that an SM has 32 warps, against 74 and 24: 90 us with gelu, though
// bf16 spills 48 bytes a thread so (f16 none).
#include <algorithm>

#include "column_sum.cuh"
#include "vec8.cuh"

namespace tpg {
namespace {

constexpr int kPer = 8;                  // columns of a thread
constexpr int kThreads = 256;
constexpr int kWide = 64, kNarrow = 8;   // threads side by side in a block

template <typename T, int ACT, int SIDE>
__device__ __forceinline__ void act_grad_strip(const ActGradOp& op, int strips, bool vec,
                                               float (&sum)[kPer]) {
    const int t = threadIdx.x % SIDE, lane_row = threadIdx.x / SIDE;
    const int64_t n = (int64_t(blockIdx.x) * SIDE + t) * kPer;
    const int64_t m_begin = op.M * blockIdx.y / strips, m_end = op.M * (blockIdx.y + 1) / strips;
    if (n >= op.N) return;
    const int cnt = op.N - n < kPer ? int(op.N - n) : kPer;
    vec = vec && cnt == kPer;
    constexpr bool kAct = ACT != TPGEMM_ACT_NONE;
    constexpr int kStep = kThreads / SIDE;
    const auto row = [&](int64_t m, float (&dd)[8], const float (&z)[8]) {
        if constexpr (kAct) {
#pragma unroll
            for (int j = 0; j < 8; j += 2)
                split(mul(f2(dd[j], dd[j + 1]), act_bwd<ACT>(f2(z[j], z[j + 1]))), dd[j], dd[j + 1]);
            // The two products read dZ in the operands' own type.
            if (op.dZ) store8<T>(op.dZ, m * op.lddz + n, vec, cnt, dd);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += dd[j];
    };
    if (vec) {
        // kAhead rows' loads are under way while one is computed.
        constexpr int kAhead = kAct ? 2 : 4;
        const T* pd = static_cast<const T*>(op.dY) + n;
        const T* pz = static_cast<const T*>(op.Z) + n;
        uint4 rd[kAhead], rz[kAhead];
        const auto fetch = [&](int i, int64_t m) {
            if (m >= m_end) return;
            rd[i] = *reinterpret_cast<const uint4*>(pd + m * op.lddy);
            if constexpr (kAct) rz[i] = *reinterpret_cast<const uint4*>(pz + m * op.ldz);
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) fetch(i, m_begin + lane_row + i * kStep);
        for (int64_t m = m_begin + lane_row; m < m_end; m += kAhead * kStep) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int64_t at = m + i * kStep;
                if (at >= m_end) break;
                float dd[8], z[8];
                unpack8<T>(rd[i], dd);
                if constexpr (kAct) unpack8<T>(rz[i], z);
                fetch(i, at + kAhead * kStep);
                row(at, dd, z);
            }
        }
        return;
    }
    for (int64_t m = m_begin + lane_row; m < m_end; m += kStep) {
        float dd[8], z[8];
        load8<T>(op.dY, m * op.lddy + n, false, cnt, dd);
        if constexpr (kAct) load8<T>(op.Z, m * op.ldz + n, false, cnt, z);
        row(m, dd, z);
    }
}

template <typename T, int SIDE>
__global__ void __launch_bounds__(kThreads, 4)
    act_grad_kernel(const __grid_constant__ ActGradOp op, int strips, bool vec) {
    constexpr int kRows = kThreads / SIDE, kCols = SIDE * kPer;
    __shared__ float s[kRows][kCols];
    grid_launch_dependents();
    grid_dependency_wait();
    float sum[kPer] = {};
    with_act(op.act, [&](auto act) {
        act_grad_strip<T, decltype(act)::value, SIDE>(op, strips, vec, sum);
    });
    if (!op.dbias) return;
    const int t = threadIdx.x % SIDE, lane_row = threadIdx.x / SIDE;
#pragma unroll
    for (int j = 0; j < kPer; ++j) s[lane_row][j * SIDE + t] = sum[j];
    __syncthreads();
    for (int c = threadIdx.x; c < kCols; c += kThreads) {
        const int64_t n = int64_t(blockIdx.x) * kCols + c;
        if (n >= op.N) continue;
        const int at = (c % kPer) * SIDE + c / kPer;
        float v = 0.f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) v += s[r][at];
        if (SIDE == kWide)
            op.partial[int64_t(blockIdx.y) * op.N + n] = v;
        else if (op.grad == TPGEMM_ELEM_F32)
            static_cast<float*>(op.dbias)[n] = v;
        else if (op.grad == TPGEMM_ELEM_BF16)
            static_cast<__nv_bfloat16*>(op.dbias)[n] = from_f32<__nv_bfloat16>(v);
        else
            static_cast<__half*>(op.dbias)[n] = from_f32<__half>(v);
    }
}

// The gated layer's: Z holds gates g and factors u, N columns of each, and
//   dZ[m, n] = dY u act'(g),  dZ[m, N + n] = dY act(g),
// with the sums of both. A thread takes eight outputs, from dY and both halves of
// Z, which it copies kGatedAhead rows ahead to its own places in shared memory (silu
// of 4096 x 4096 bf16, dbias alone: 24 us so, 35 with one row ahead in registers).
//
// A 32-bit dW takes dZ as two 16-bit values, its rounding and what that left (REST):
// from the rounding alone it would be off by 2^-9 (bf16) or 2^-12 (f16) of its
// terms. The rest of an f16 value may lie below f16's normal numbers, so it is kept
// 2^11 times as large, which fits f16 for every rounding that does. Activations are
// then those of 32-bit results (FINE), and so for a 32-bit dbias: gelu's other form is
// off by up to 1e-4 of itself, ten times what the two values of dZ lose (dbias alone of
// 4096 x 4096 with gelu 31 us, 29 with that form).
constexpr int kGatedAhead = 3;
using GatedRing = uint4[kGatedAhead][3][kThreads];

template <typename T>
constexpr float kRestScale = std::is_same<T, __half>::value ? 1.f / 2048.f : 1.f;

template <typename T>
__device__ __forceinline__ void rest_of(const float (&x)[8], float (&low)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float high = to_f32(from_f32<T>(x[j]));
        low[j] = isinf(high) ? 0.f : (x[j] - high) * (1.f / kRestScale<T>);  // (a NaN stays one)
    }
}

template <typename T, int ACT, int SIDE, bool REST, bool FINE>
__device__ __forceinline__ void gated_grad_strip(const ActGradOp& op, void* rest, int strips, bool vec,
                                                 GatedRing& ring, float (&sg)[kPer], float (&su)[kPer]) {
    const int t = threadIdx.x % SIDE, lane_row = threadIdx.x / SIDE;
    const int64_t n = (int64_t(blockIdx.x) * SIDE + t) * kPer;
    const int64_t m_begin = op.M * blockIdx.y / strips, m_end = op.M * (blockIdx.y + 1) / strips;
    if (n >= op.N) return;
    const int cnt = op.N - n < kPer ? int(op.N - n) : kPer;
    vec = vec && cnt == kPer;
    constexpr int kStep = kThreads / SIDE;
    const auto row = [&](int64_t m, const float (&dy)[8], const float (&g)[8], const float (&u)[8]) {
        float dg[8], du[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const F2 z = f2(g[j], g[j + 1]), d = f2(dy[j], dy[j + 1]);
            split(mul(mul(d, f2(u[j], u[j + 1])), act_bwd<ACT, FINE>(z)), dg[j], dg[j + 1]);
            split(mul(d, act_fwd<ACT, FINE>(z)), du[j], du[j + 1]);
        }
        // The two products read dZ in the operands' own type.
        if (op.dZ) {
            store8<T>(op.dZ, m * op.lddz + n, vec, cnt, dg);
            store8<T>(op.dZ, m * op.lddz + op.N + n, vec, cnt, du);
        }
        if constexpr (REST) {
            float low[8];
            rest_of<T>(dg, low);
            store8<T>(rest, m * op.lddz + n, vec, cnt, low);
            rest_of<T>(du, low);
            store8<T>(rest, m * op.lddz + op.N + n, vec, cnt, low);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sg[j] += dg[j];
            su[j] += du[j];
        }
    };
    if (vec) {
        const T* pd = static_cast<const T*>(op.dY) + n;
        const T* pz = static_cast<const T*>(op.Z) + n;
        const auto fetch = [&](int slot, int64_t m) {
            if (m < m_end) {
                cp_async_16(smem_u32(&ring[slot][0][threadIdx.x]), pd + m * op.lddy, 16);
                cp_async_16(smem_u32(&ring[slot][1][threadIdx.x]), pz + m * op.ldz, 16);
                cp_async_16(smem_u32(&ring[slot][2][threadIdx.x]), pz + m * op.ldz + op.N, 16);
            }
            cp_async_commit();
        };
        int64_t m = m_begin + lane_row;
#pragma unroll
        for (int i = 0; i < kGatedAhead; ++i) fetch(i, m + i * kStep);
        for (int slot = 0; m < m_end; m += kStep, slot = slot + 1 == kGatedAhead ? 0 : slot + 1) {
            cp_async_wait<kGatedAhead - 1>();
            float dy[8], g[8], u[8];
            unpack8<T>(ring[slot][0][threadIdx.x], dy);
            unpack8<T>(ring[slot][1][threadIdx.x], g);
            unpack8<T>(ring[slot][2][threadIdx.x], u);
            fetch(slot, m + kGatedAhead * kStep);
            row(m, dy, g, u);
        }
        cp_async_wait<0>();
        return;
    }
    for (int64_t m = m_begin + lane_row; m < m_end; m += kStep) {
        float dy[8], g[8], u[8];
        load8<T>(op.dY, m * op.lddy + n, false, cnt, dy);
        load8<T>(op.Z, m * op.ldz + n, false, cnt, g);
        load8<T>(op.Z, m * op.ldz + op.N + n, false, cnt, u);
        row(m, dy, g, u);
    }
}

template <typename T, int SIDE, bool REST, bool FINE>
__global__ void __launch_bounds__(kThreads, 3)
    gated_grad_kernel(const __grid_constant__ ActGradOp op, const DzRest rest, int strips, bool vec) {
    constexpr int kRows = kThreads / SIDE, kCols = SIDE * kPer;
    __shared__ union {
        GatedRing ring;
        float s[kRows][2][kCols];
    } shared;
    auto& s = shared.s;
    grid_launch_dependents();
    grid_dependency_wait();
    float sg[kPer] = {}, su[kPer] = {};
    with_act(op.act, [&](auto act) {
        gated_grad_strip<T, decltype(act)::value, SIDE, REST, FINE>(op, rest.low, strips, vec, shared.ring, sg, su);
    });
    if constexpr (REST) {
        if (blockIdx.y == 0)
            for (int i = threadIdx.x; i < 2 * kCols; i += kThreads) {
                const int64_t n = int64_t(blockIdx.x) * kCols + i % kCols;
                if (n < op.N) rest.scale[n + (i / kCols) * op.N] = kRestScale<T>;
            }
    }
    if (!op.dbias) return;
    __syncthreads();  // (the ring's place)
    const int t = threadIdx.x % SIDE, lane_row = threadIdx.x / SIDE;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        s[lane_row][0][j * SIDE + t] = sg[j];
        s[lane_row][1][j * SIDE + t] = su[j];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * kCols; i += kThreads) {
        const int h = i / kCols, c = i % kCols;
        int64_t n = int64_t(blockIdx.x) * kCols + c;
        if (n >= op.N) continue;
        n += h * op.N;
        const int at = (c % kPer) * SIDE + c / kPer;
        float v = 0.f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) v += s[r][h][at];
        if (SIDE == kWide)
            op.partial[int64_t(blockIdx.y) * 2 * op.N + n] = v;
        else if (op.grad == TPGEMM_ELEM_F32)
            static_cast<float*>(op.dbias)[n] = v;
        else if (op.grad == TPGEMM_ELEM_BF16)
            static_cast<__nv_bfloat16*>(op.dbias)[n] = from_f32<__nv_bfloat16>(v);
        else
            static_cast<__half*>(op.dbias)[n] = from_f32<__half>(v);
    }
}

// Rows of `bytes` bytes, `pitch` apart and anywhere in memory, to rows of whole
// 16-byte units; a thread to a unit, blockIdx.z to a matrix. A unit with another
// one behind it in its row is read as five aligned words and shifted into place,
// the last one or two byte by byte, and so the matrix's first one where its first
// word begins before it.
__global__ void __launch_bounds__(256) align_rows_kernel(const __grid_constant__ AlignJobs jobs) {
    grid_launch_dependents();
    grid_dependency_wait();
    const AlignJob& job = jobs.j[blockIdx.z];
    const int64_t u = int64_t(blockIdx.x) * 32 + (threadIdx.x & 31);
    const int64_t bytes = job.bytes;
    if (16 * u >= bytes) return;
#pragma unroll 4
    for (int64_t r = int64_t(blockIdx.y) * 8 + (threadIdx.x >> 5); r < job.rows; r += int64_t(gridDim.y) * 8) {
        const uint8_t* p = job.src + r * job.pitch + 16 * u;
        uint32_t w[4] = {};
        const uint32_t off = uint32_t(reinterpret_cast<uintptr_t>(p) & 3u);
        if (16 * u + 32 <= bytes && p - off >= job.src) {
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
        *reinterpret_cast<uint4*>(job.dst + r * job.dst_pitch + 16 * u) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

}  // namespace

// One strip up to kFewRows rows (100 x 520 f16: 3.5 us, 5.1 in two launches;
// 256 x 4096: 5.7 and 7.2; 256 x 520, where few blocks have all the rows: 5.6
// and 5.1);
// else enough that the blocks fill the GPU about four times over, of at least
// 16 rows each.
constexpr int64_t kFewRows = 256;

int act_grad_strips(int64_t M, int64_t N) {
    if (M <= kFewRows) return 1;
    const int64_t cb = (N + kWide * kPer - 1) / (kWide * kPer);
    const int64_t want = cb > 0 ? (4 * kSms + cb - 1) / cb : 1;
    const int64_t most = (M + 15) / 16;
    return int(want < most ? want : most);
}

cudaError_t launch_act_grad(const ActGradOp& op, cudaStream_t stream) {
    const int strips = act_grad_strips(op.M, op.N);
    const bool few = strips == 1;
    const int cols = (few ? kNarrow : kWide) * kPer;
    const int64_t cb = (op.N + cols - 1) / cols;
    if (cb > 0x7fffffff || strips > 65535) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(cb), static_cast<unsigned>(strips));
    auto rows16 = [&](const void* p, int64_t ld) {
        return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (op.M <= 1 || ld % 8 == 0));
    };
    const bool vec = rows16(op.dY, op.lddy) && rows16(op.Z, op.ldz) && rows16(op.dZ, op.lddz);
    const bool f16 = op.dtype == TPGEMM_ELEM_F16;
    auto fn = few ? (f16 ? act_grad_kernel<__half, kNarrow> : act_grad_kernel<__nv_bfloat16, kNarrow>)
                  : (f16 ? act_grad_kernel<__half, kWide> : act_grad_kernel<__nv_bfloat16, kWide>);
    const cudaError_t e = launch_dependent(fn, grid, dim3(kThreads), 0, stream, op, strips, vec);
    if (e != cudaSuccess || !op.dbias || few) return e;
    return launch_column_sum(op.partial, strips, op.N, op.dbias, op.grad, stream);
}

int gated_grad_strips(int64_t M, int64_t N) { return act_grad_strips(M, N); }

template <typename T, bool REST, bool FINE>
static cudaError_t launch_gated_typed(const ActGradOp& op, const DzRest& rest, cudaStream_t stream) {
    const int strips = gated_grad_strips(op.M, op.N);
    const bool few = strips == 1;
    const int cols = (few ? kNarrow : kWide) * kPer;
    const int64_t cb = (op.N + cols - 1) / cols;
    if (cb > 0x7fffffff || strips > 65535) return cudaErrorInvalidValue;
    auto rows16 = [&](const void* p, int64_t ld) {
        return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (op.M <= 1 || ld % 8 == 0));
    };
    const bool vec = op.N % 8 == 0 && rows16(op.dY, op.lddy) && rows16(op.Z, op.ldz) && rows16(op.dZ, op.lddz);
    auto fn = few ? gated_grad_kernel<T, kNarrow, REST, FINE> : gated_grad_kernel<T, kWide, REST, FINE>;
    const cudaError_t e = launch_dependent(fn, dim3(unsigned(cb), unsigned(strips)), dim3(kThreads), 0, stream, op,
                                           rest, strips, vec);
    if (e != cudaSuccess || !op.dbias || few) return e;
    return launch_column_sum(op.partial, strips, 2 * op.N, op.dbias, op.grad, stream);
}

template <typename T>
static cudaError_t launch_gated_of(const ActGradOp& op, const DzRest& rest, cudaStream_t stream) {
    if (op.grad != TPGEMM_ELEM_F32) return launch_gated_typed<T, false, false>(op, rest, stream);
    return rest.low ? launch_gated_typed<T, true, true>(op, rest, stream)
                    : launch_gated_typed<T, false, true>(op, rest, stream);
}

cudaError_t launch_gated_grad(const ActGradOp& op, const DzRest& rest, cudaStream_t stream) {
    return op.dtype == TPGEMM_ELEM_F16 ? launch_gated_of<__half>(op, rest, stream)
                                       : launch_gated_of<__nv_bfloat16>(op, rest, stream);
}

constexpr int64_t kAlignBlocks = 8 * kSms;  // eight to an SM; a warp then has several rows' loads in flight

cudaError_t launch_align_rows(const AlignJobs& jobs, cudaStream_t stream) {
    if (jobs.n == 0) return cudaSuccess;
    int64_t bx = 1, by = 1;
    for (int i = 0; i < jobs.n; ++i) {
        bx = std::max(bx, (jobs.j[i].bytes + 511) / 512);
        by = std::max(by, (jobs.j[i].rows + 7) / 8);
    }
    if (bx > 0x7fffffff) return cudaErrorInvalidValue;
    by = std::min(by, std::max<int64_t>(1, kAlignBlocks / bx));
    return launch_dependent(align_rows_kernel, dim3(unsigned(bx), unsigned(by), unsigned(jobs.n)), dim3(256),
                            0, stream, jobs);
}

}  // namespace tpg
