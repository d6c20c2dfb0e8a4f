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
// A row is read once, by a team of threads (a warp for narrow rows, up to a block),
// 16 bytes to a thread at a time. Blocks stay and walk the rows; each thread copies
// its own columns of the rows to come to its own places in shared memory (cp.async),
// where they wait without holding registers and without a barrier, so that memory is
// kept busy through a row's reductions. Rows that start anywhere are copied in
// aligned 16 bytes and joined; rows wider than a team's registers (16384 columns) are
// kept in shared memory as far as it goes, the rest read again for each pass.
//
// 8192 x 4096 bf16 with residual 48 us (83 % of memory's rate), with dropout 54
// (74 %); gradients with dh 47 (85 %) and 65 (77 %). 172 and 287 instructions to eight
// columns, gradients 192 and 318. With dropout it is not issue that bounds them (55 % of
// the slots are used) but the random words' products, whose pipe is busy for 60 % of the
// time, and the waits for it, for shared memory and at barriers between, which 27 warps
// to an SM (gradients 15) do not hide. Rows that start anywhere take some 610 to eight
// columns: 4096 x 4099 55 us, gradients 82.
#pragma once

#include <algorithm>

#include "column_sum.cuh"
#include "launch.cuh"
#include "norm_rows.cuh"
#include "philox.cuh"
#include "windows.h"

namespace tpg {
namespace {

// Sums of a and b over the block through `s`. (Reductions that follow one another
// take different `s`; the one before last may be used again.)
__device__ __forceinline__ void block_sum(float& a, float& b, float2* s) {
    const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
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

// Dropout of a thread's group but for the factor; the whole warp calls it.
template <bool VEC>
__device__ __forceinline__ void keep_cols(const Drop& d, const DropRow& w, const Cols<VEC>& c, float (&x)[8]) {
    if constexpr (VEC) {
        if (c.n == 8) {
            keep4(d, w, uint32_t(c.first / 4), x);
            keep4(d, w, uint32_t(c.first / 4 + 1), x + 4);
        }
    } else {
        keep8_apart(d, w, c.first, c.step, x);
    }
}

template <typename XT, bool VEC, bool DROP>
__device__ __forceinline__ void load_sum(const LayerNormOp& op, const DropRow& w, int64_t row, const Cols<VEC>& c,
                                         float (&h)[8]) {
    load_cols<XT, VEC>(op.X, row * op.ldx, c, h);
    if constexpr (DROP) keep_cols<VEC>(op.drop, w, c, h);
    const float scale = DROP ? op.drop.scale : 1.f;
    if (op.R) {
        float r[8];
        load_cols<XT, VEC>(op.R, row * op.ldr, c, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = fmaf(h[j], scale, r[j]);
    } else if constexpr (DROP) {
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] *= scale;
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
__device__ __forceinline__ Stats stats_of(float mean, float d, float dd, float inv_n, float eps) {
    const float off = d * inv_n;
    float var = fmaf(dd, inv_n, -off * off);
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

// ------------------------------------------------------------ aligned rows
// A team takes a row in pieces of 16 bytes: piece i of thread t holds the columns from
// kCols (i threads + t) on, so that a warp's accesses are contiguous.
template <typename T>
constexpr int kCols = 16 / int(sizeof(T));

// Where rows lie: anywhere; on 16-byte boundaries, in whole pieces; and then with
// all of a team's pieces in the row.
enum Rows { kAnywhere, kAligned, kWhole };

__device__ __forceinline__ int off16(const void* p) { return int(reinterpret_cast<uintptr_t>(p) & 15u); }

// Places for rows to come: `depth` rows of `inputs` matrices, P pieces each. Of
// aligned rows only the thread itself writes and reads its places, so no barrier is
// needed. Of others a piece's place holds the aligned 16 bytes that it starts in, and
// the piece is joined from there and the next lane's place; a place more for each warp
// holds the bytes behind its last lane's. (Bytes before a row's start are read with
// those of its 16, but not those before the matrix or behind a row's end.)
template <typename T, int P, int STEP, int ROWS>  // STEP: threads that places are laid out for
struct Ring {
    uint4* base;
    int inputs, depth;
    __device__ __forceinline__ Ring(void* smem, int depth, int inputs)
        : base(static_cast<uint4*>(smem)), inputs(inputs), depth(depth) {}
    static constexpr int kSpare = ROWS == kAnywhere ? STEP / 32 : 0;
    __device__ __forceinline__ uint4* row(int slot) const { return base + slot * inputs * P * (STEP + kSpare) + threadIdx.x; }
    __device__ __forceinline__ static int place(int input, int piece) { return (input * P + piece) * (STEP + kSpare); }
    // The warp's spare place.
    __device__ __forceinline__ static int spare(int input, int piece) {
        return place(input, piece) + STEP + int(threadIdx.x >> 5) - int(threadIdx.x);
    }
    // The piece at column c of the row of `cols` columns at p, of the matrix at `base`; the
    // whole warp calls it. FIRST: p may be one of the matrix's first eight rows, of which
    // short ones may all start in the 16 bytes that the matrix does.
    template <bool FIRST>
    __device__ __forceinline__ void fetch(uint4* row, int input, int piece, const void* base, const T* p, int c,
                                          int cols) const {
        if constexpr (ROWS != kAnywhere) {
            cp_async_16(smem_u32(row + place(input, piece)), p + c, 16);
        } else {
            const uintptr_t at = reinterpret_cast<uintptr_t>(p);
            const uint64_t bytes = uint64_t(cols) * sizeof(T), offset = uint64_t(c) * sizeof(T);
            const CopyWindow w = copy_window(at, bytes, offset);
            if (FIRST && piece == 0 && begins_apart(at, reinterpret_cast<uintptr_t>(base), offset))
                row[place(input, 0)] = load_window(reinterpret_cast<const uint8_t*>(p), -int64_t(at & 15), int64_t(bytes));
            else
                cp_async_16(smem_u32(row + place(input, piece)), reinterpret_cast<const void*>(w.at), w.bytes);
            if ((threadIdx.x & 31) == 31) {
                const CopyWindow v = copy_window(at, bytes, offset + 16);
                cp_async_16(smem_u32(row + spare(input, piece)), reinterpret_cast<const void*>(v.at), v.bytes);
            }
        }
    }
    // off: off16 of the row. Columns past the row are zero.
    __device__ __forceinline__ void get(const uint4* row, int input, int piece, int off, F2 (&f)[kPairs<T>]) const {
        uint4 v = row[place(input, piece)];
        if constexpr (ROWS == kAnywhere)
            v = join_windows(v, row[(threadIdx.x & 31) == 31 ? spare(input, piece) : place(input, piece) + 1], off);
        unpack_pairs<T>(v, f);
    }
    // The oldest of `depth` rows in flight (a group of copies each) has arrived.
    __device__ __forceinline__ void wait() const {
        switch (depth) {
            case 1: cp_async_wait<0>(); break;
            case 2: cp_async_wait<1>(); break;
            case 3: cp_async_wait<2>(); break;
            default: cp_async_wait<3>(); break;
        }
        pass_on();
    }
    // Before a lane reads what others copied, and before it copies over what they read.
    __device__ __forceinline__ void pass_on() const {
        if constexpr (ROWS == kAnywhere) __syncwarp();
    }
};
constexpr int kMaxDepth = 4;

// Threads of a block of teams of any size: 640 of the norm's, which have 96 registers
// each then, take more of the teams that do not fill 512 (bf16 4096 x 4099 57 us, 63
// with 512 threads; 8192 x 2560 31 and 37, 4096 x 6144 34 and 38, f32 4096 x 4099 107
// and 151), at the price of rows of which as many fit 512 (4096 x 7168 with dropout 62
// and 58). Eight pieces to a thread want more registers (f32 2048 x 12301 217 and 207),
// and the gradients do (4096 x 5120 70 and 57).
constexpr int any_threads(int pieces, bool grad) { return grad || pieces > 4 ? 512 : 640; }

// A spread of rows: P pieces to a thread of a team of T threads (T = 0: any team). T
// is a constant where the row is whole and T a power of two, since places and
// addresses then are: 8192 x 4096 bf16 with dropout takes 55 us so, 62 otherwise. Threads of a block at most, and
// blocks to an SM at least, by the registers that a thread then has: the norm does
// with 64, the gradients, which hold two sums for each column, with 128.
template <int P, int T, bool GRAD>
struct RowKernel {
    static constexpr int kThreads = T == 0 ? any_threads(P, GRAD) : GRAD && T <= 256 ? 256 : 512;
    static constexpr int kBlocks = T == 0 || (GRAD && T == 512) ? 1 : 2;
};

// How the rows of a call are spread (ring_plan): threads of a team, rows that a
// thread copies ahead, and where behind them the weights lie (0: they are not held).
struct RingPlan {
    int team, depth, weights_at;
};

// Gamma and beta, of XT or 32-bit: held in shared memory behind the ring, for all
// teams of a block (from L2 they would come in the midst of every row), or, of rows
// too wide for that, read from memory. WIDE: held as 32-bit values.
template <typename XT, int P, int ROWS, bool WIDE>
struct Weights {
    uint4* mine;     // the thread's first place; null: not held
    int elem, step;  // their type in memory, and 16-byte units between a thread's places
    int cols;
    // Units of a piece's columns.
    template <typename T>
    static constexpr int kUnits = kCols<XT> / kCols<T>;
    // 16 bytes from column c on, zero past the last column.
    template <typename T>
    __device__ __forceinline__ uint4 load(const T* p, int c) const {
        if constexpr (ROWS != kAnywhere) return *reinterpret_cast<const uint4*>(p + c);
        uint32_t w[4] = {};
#pragma unroll
        for (int i = 0; i < kCols<T>; ++i) {
            if (c + i >= cols) break;
            if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(p[c + i]);
            else w[i / 2] |= uint32_t(reinterpret_cast<const uint16_t*>(p)[c + i]) << (16 * (i & 1));
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    template <typename T>
    __device__ __forceinline__ void get_as(int which, int piece, const void* p, int c, F2 (&f)[kPairs<XT>]) const {
        const bool here = mine && (!WIDE || sizeof(T) == 4);
#pragma unroll
        for (int u = 0; u < kUnits<T>; ++u) {
            const uint4 v = here ? mine[((which * P + piece) * kUnits<T> + u) * step]
                                 : load(static_cast<const T*>(p), c + u * kCols<T>);
            F2 part[kPairs<T>];
            unpack_pairs<T>(v, part);
#pragma unroll
            for (int j = 0; j < kPairs<T>; ++j) f[u * kPairs<T> + j] = part[j];
        }
    }
    __device__ __forceinline__ void get(int which, int piece, const void* p, int c, F2 (&f)[kPairs<XT>]) const {
        if (elem == TPGEMM_ELEM_F32 || (WIDE && mine)) get_as<float>(which, piece, p, c, f);
        else get_as<XT>(which, piece, p, c, f);
    }
    template <typename T>
    __device__ __forceinline__ void hold_as(int which, int piece, const void* p, int c) const {
        if constexpr (WIDE && sizeof(T) == 2) {
            F2 f[kPairs<T>];
            unpack_pairs<T>(load(static_cast<const T*>(p), c), f);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const F2 two[2] = {f[2 * u], f[2 * u + 1]};
                store_pairs(reinterpret_cast<float*>(mine + ((which * P + piece) * 2 + u) * step), two);
            }
        } else {
#pragma unroll
            for (int u = 0; u < kUnits<T>; ++u)
                mine[((which * P + piece) * kUnits<T> + u) * step] = load(static_cast<const T*>(p), c + u * kCols<T>);
        }
    }
    // By one team.
    __device__ __forceinline__ void hold(int which, int piece, const void* p, int c) const {
        if (elem == TPGEMM_ELEM_F32) hold_as<float>(which, piece, p, c);
        else hold_as<XT>(which, piece, p, c);
    }
};

// The threads that share a row: T of them, or `any` (a multiple of 32); `first` is the
// block's number of the team's first warp, t a thread's place.
template <int T>
struct Team {
    int any, first, index, t;
    __device__ __forceinline__ explicit Team(int any) : any(any) {
        index = int(threadIdx.x) / threads();
        first = index * warps();
        t = int(threadIdx.x) - index * threads();
    }
    __device__ __forceinline__ int threads() const { return T ? T : any; }
    __device__ __forceinline__ int warps() const { return threads() / 32; }
    // (Barriers 1 and up; 0 is the block's.)
    __device__ __forceinline__ void sync() const {
        asm volatile("bar.sync %0, %1;" ::"r"(1 + index), "r"(threads()) : "memory");
    }
    __device__ __forceinline__ int halves() const {  // the largest power of two below warps()
        return T ? T / 64 : 1 << (31 - __clz(warps() - 1));
    }
    // Sums of N values over the team, through `s`, a place of the block's warps that
    // the reduction before last may have used.
    template <int N>
    __device__ __forceinline__ void sum(float (&a)[N], float2* s) const {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) a[i] += __shfl_xor_sync(0xffffffffu, a[i], o);
        if (warps() == 1) return;
        const int lane = threadIdx.x & 31;
        if (lane == 0) s[threadIdx.x >> 5] = make_float2(a[0], a[N - 1]);
        sync();
        const float2 v = lane < warps() ? s[first + lane] : make_float2(0.f, 0.f);
        a[0] = v.x;
        a[N - 1] = N > 1 ? v.y : v.x;
#pragma unroll
        for (int o = halves(); o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) a[i] += __shfl_xor_sync(0xffffffffu, a[i], o);
#pragma unroll
        for (int i = 0; i < N; ++i) a[i] = __shfl_sync(0xffffffffu, a[i], 0);
    }
    __device__ __forceinline__ uint32_t max(uint32_t v, float2* s) const {
        v = __reduce_max_sync(0xffffffffu, v);
        if (warps() == 1) return v;
        const int lane = threadIdx.x & 31;
        if (lane == 0) s[threadIdx.x >> 5].x = __uint_as_float(v);
        sync();
        return __reduce_max_sync(0xffffffffu, lane < warps() ? __float_as_uint(s[first + lane].x) : 0u);
    }
};

template <int N>
__device__ __forceinline__ void zero(F2 (&f)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = f2(0.f);
}

template <int N>
__device__ __forceinline__ float sum_of(const F2 (&f)[N]) {
    F2 v = add(f[0], f[1]);
    if constexpr (N == 4) v = add(v, add(f[2], f[3]));
    float a, b;
    split(v, a, b);
    return a + b;
}

// Dropout of 2 N neighbouring elements from column c on, but for the factor.
template <int N>
__device__ __forceinline__ void keep_pairs(const Drop& d, const DropRow& w, int c, F2 (&f)[N]) {
    float x[2 * N];
#pragma unroll
    for (int i = 0; i < N; ++i) split(f[i], x[2 * i], x[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) keep4(d, w, uint32_t(c) / 4 + i, x + 4 * i);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = f2(x[2 * i], x[2 * i + 1]);
}

// Zeroes all but the first n of 2 N values.
template <int N>
__device__ __forceinline__ void keep_first(int n, F2 (&f)[N]) {
    if (n >= 2 * N) return;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float a, b;
        split(f[i], a, b);
        f[i] = f2(2 * i < n ? a : 0.f, 2 * i + 1 < n ? b : 0.f);
    }
}

template <typename U>
__device__ __forceinline__ U part_of(const uint4& v, int i) {  // (i a constant)
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (sizeof(U) == 4) return w[i];
    else return U(w[i / 2] >> (16 * (i & 1)));
}

// Stores 16 bytes of neighbouring elements from each lane, the first n of a lane's, to
// rows that start anywhere: each lane the aligned 16 bytes that its own begin in, with
// the end of the lane's before it, and the warp's two ends element by element. The
// whole warp calls it; all lanes before one that has elements are full.
template <typename O, int N>
__device__ __forceinline__ void store_anywhere(O* p, int n, const F2 (&f)[N]) {
    if constexpr (2 * N * sizeof(O) != 16) {
        float x[2 * N];
#pragma unroll
        for (int i = 0; i < N; ++i) split(f[i], x[2 * i], x[2 * i + 1]);
#pragma unroll
        for (int i = 0; i < 2 * N; ++i)
            if (i < n) p[i] = from_f32<O>(x[i]);
    } else {
        using U = typename std::conditional<sizeof(O) == 4, uint32_t, uint16_t>::type;
        constexpr int kSize = int(sizeof(O));
        uint4 v;
        store_pairs(reinterpret_cast<O*>(&v), f);
        const int lane = threadIdx.x & 31, off = off16(p);
        const Window before = make_uint4(__shfl_up_sync(0xffffffffu, v.x, 1), __shfl_up_sync(0xffffffffu, v.y, 1),
                                         __shfl_up_sync(0xffffffffu, v.z, 1), __shfl_up_sync(0xffffffffu, v.w, 1));
        const int n_before = __shfl_up_sync(0xffffffffu, n, 1);
        const uint4 w = off ? join_windows(before, v, 16 - off) : v;
        // This lane's window of 16 bytes holds elements [lo, hi) of the row.
        const int skip = off / kSize;
        int lo = lane == 0 ? skip : 0;
        int hi = n > 0 ? min(2 * N, skip + n) : lane > 0 ? n_before - (2 * N - skip) : 0;
        U* q = reinterpret_cast<U*>(reinterpret_cast<uint8_t*>(p) - off);
        if (lo == 0 && hi == 2 * N) {
            *reinterpret_cast<uint4*>(q) = w;
            lo = hi = 0;
        }
        // What is left: parts of windows, and the start of the window behind the last
        // lane's, whose own is then a whole one.
        uint4 rest = w;
        if (lane == 31 && skip && n > 2 * N - skip) {
            lo = 2 * N - skip;
            hi = n;
            q = reinterpret_cast<U*>(p);
            rest = v;
        }
        if (lo < hi) {
            const uint32_t mask = ((1u << hi) - 1u) & ~((1u << lo) - 1u);
#pragma unroll
            for (int i = 0; i < 2 * N; ++i)
                if ((mask >> i) & 1u) q[i] = part_of<U>(rest, i);
        }
    }
}

template <int ROWS, typename O, int N>
__device__ __forceinline__ void store_piece(O* p, int n, const F2 (&f)[N]) {
    if constexpr (ROWS == kAnywhere) store_anywhere(p, n, f);
    else store_pairs(p, f);
}

template <typename XT, int P, int T, int ROWS, bool DROP>
__global__ void __launch_bounds__(RowKernel<P, T, false>::kThreads, RowKernel<P, T, false>::kBlocks)
    layernorm_rows_kernel(const __grid_constant__ LayerNormOp op, const RingPlan plan) {
    constexpr int N = kPairs<XT>;
    extern __shared__ __align__(16) uint8_t ring_smem[];
    __shared__ float2 s[3][32];
    const Team<T> team(plan.team);
    const int64_t teams = blockDim.x / unsigned(team.threads()), stride = gridDim.x * teams;
    int64_t row = blockIdx.x * teams + team.index;
    const int cols = int(op.cols), depth = plan.depth;
    const Ring<XT, P, RowKernel<P, T, false>::kThreads, ROWS> ring(ring_smem, depth, op.R ? 2 : 1);
    const Weights<XT, P, ROWS, false> weights{
        plan.weights_at ? reinterpret_cast<uint4*>(ring_smem + plan.weights_at) + team.t : nullptr, op.g, team.threads(), cols};
    const auto column = [&](int i) { return kCols<XT> * (i * team.threads() + team.t); };
    // Whether piece i is in the row (of rows anywhere: the warp's first lane's is), and its columns there.
    const auto has = [&](int i) {
        return ROWS == kWhole || column(i) - (ROWS == kAnywhere ? kCols<XT> * int(threadIdx.x & 31) : 0) < cols;
    };
    const auto count = [&](int i) { return ROWS == kAnywhere ? max(0, min(kCols<XT>, cols - column(i))) : kCols<XT>; };
    // (first: whether r may be one of the first eight rows, a constant. Blocks' later rows
    // are not: a turn of the grid takes all rows, or 152 and more.)
    const auto fetch = [&](int64_t r, uint4* place, auto first) {
        constexpr bool kFirst = decltype(first)::value;
        if (r < op.rows) {
            const XT* x = static_cast<const XT*>(op.X) + r * op.ldx;
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (has(i)) ring.template fetch<kFirst>(place, 0, i, op.X, x, column(i), cols);
            if (op.R) {
                const XT* q = static_cast<const XT*>(op.R) + r * op.ldr;
#pragma unroll
                for (int i = 0; i < P; ++i)
                    if (has(i)) ring.template fetch<kFirst>(place, 1, i, op.R, q, column(i), cols);
            }
        }
        cp_async_commit();
    };
    grid_launch_dependents();
    grid_dependency_wait();
    if (ROWS == kAnywhere) fetch(row, ring.row(0), std::true_type());
    for (int i = ROWS == kAnywhere; i < depth; ++i) fetch(row + i * stride, ring.row(i), std::false_type());
    if (weights.mine) {
        if (team.index == 0)
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (has(i)) {
                    weights.hold(0, i, op.gamma, column(i));
                    if (op.beta) weights.hold(1, i, op.beta, column(i));
                }
        if (teams > 1) __syncthreads();  // (else each thread reads its own)
    }
    DropOffset offset{};
    if constexpr (DROP) offset = drop_offset(op.drop);
    const float inv_n = 1.f / float(op.cols);
    const F2 scale = f2(DROP ? op.drop.scale : 1.f);
    for (int slot = 0; row < op.rows; row += stride, slot = slot + 1 == depth ? 0 : slot + 1) {
        DropRow w{};
        if constexpr (DROP) w = drop_row(op.drop, offset, uint32_t(row));
        ring.wait();
        uint4* const place = ring.row(slot);
        const int off_x = off16(static_cast<const XT*>(op.X) + row * op.ldx);
        const int off_r = off16(static_cast<const XT*>(op.R) + row * op.ldr);
        F2 h[P][N];
        F2 part[N];
        zero(part);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (!has(i)) {
                zero(h[i]);
                continue;
            }
            ring.get(place, 0, i, off_x, h[i]);
            if constexpr (DROP) keep_pairs(op.drop, w, column(i), h[i]);
            F2 r[N];
            zero(r);
            if (op.R) ring.get(place, 1, i, off_r, r);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                h[i][j] = fma(h[i][j], scale, r[j]);
                part[j] = add(part[j], h[i][j]);
            }
        }
        ring.pass_on();
        fetch(row + depth * stride, place, std::false_type());
        float sum[1] = {sum_of(part)};
        team.sum(sum, s[0]);
        const float mean = sum[0] * inv_n;
        if (op.H) {
            XT* p = static_cast<XT*>(op.H) + row * op.ldh;
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (has(i)) store_piece<ROWS>(p + column(i), count(i), h[i]);
        }
        F2 d[N], dd[N];
        zero(d);
        zero(dd);
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (has(i)) {
#pragma unroll
                for (int j = 0; j < N; ++j) h[i][j] = add(h[i][j], f2(-mean));
                keep_first(count(i), h[i]);
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    d[j] = add(d[j], h[i][j]);
                    dd[j] = fma(h[i][j], h[i][j], dd[j]);
                }
            }
        float both[2] = {sum_of(d), sum_of(dd)};
        team.sum(both, s[1]);
        const Stats st = stats_of(mean, both[0], both[1], inv_n, op.eps);
        if (team.t == 0) {
            if (op.mean) op.mean[row] = st.mean + st.off;
            if (op.rstd) op.rstd[row] = st.rstd;
        }
        // y takes h's place.
        uint32_t amax = 0;
        const F2 rstd = f2(st.rstd), shift = f2(-st.off * st.rstd);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (!has(i)) continue;
            F2 g[N], b[N];
            zero(b);
            weights.get(0, i, op.gamma, column(i), g);
            if (op.beta) weights.get(1, i, op.beta, column(i), b);
#pragma unroll
            for (int j = 0; j < N; ++j) h[i][j] = fma(fma(h[i][j], rstd, shift), g[j], b[j]);
            if (op.mode == TPGEMM_SCALE_ROW) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    float lo, hi;
                    split(h[i][j], lo, hi);
                    amax = max(amax, max(abs_bits(lo), abs_bits(hi)));
                }
            }
        }
        if (op.mode == TPGEMM_SCALE_ROW) {
            const float to = row_scale(team.max(amax, s[2]), op.y);
            if (team.t == 0) op.scale[row] = to;
            const F2 inv = f2(1.f / to);
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int j = 0; j < N; ++j) h[i][j] = mul(h[i][j], inv);
        }
        const auto store = [&](auto* y) {
            y += row * op.ldy;
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (has(i)) store_piece<ROWS>(y + column(i), count(i), h[i]);
        };
        switch (op.y) {
            case TPGEMM_ELEM_F16: store(static_cast<__half*>(op.Y)); break;
            case TPGEMM_ELEM_BF16: store(static_cast<__nv_bfloat16*>(op.Y)); break;
            case TPGEMM_ELEM_E4M3: store(static_cast<e4m3*>(op.Y)); break;
            case TPGEMM_ELEM_E5M2: store(static_cast<e5m2*>(op.Y)); break;
            default: store(static_cast<float*>(op.Y)); break;
        }
    }
    cp_async_wait<0>();
}

// ---------------------------------------------------------------- wider rows
// Rows of any width, a block to a row, eight columns to a thread at a time. The first
// `held` such groups keep h in the thread's places in shared memory (49152 columns in
// all); the others are read again for each pass (2048 x 20480 bf16 with residual 130
// us, 212 with all read again).
struct Held {
    float4* mine;
    int groups;
    __device__ __forceinline__ Held(void* smem, int groups) : mine(static_cast<float4*>(smem) + threadIdx.x), groups(groups) {}
    __device__ __forceinline__ void put(int64_t i, const float (&f)[8]) const {
        if (i >= groups) return;
        float4* p = mine + i * 2 * kMaxTeam;
        p[0] = make_float4(f[0], f[1], f[2], f[3]);
        p[kMaxTeam] = make_float4(f[4], f[5], f[6], f[7]);
    }
    __device__ __forceinline__ bool get(int64_t i, float (&f)[8]) const {
        if (i >= groups) return false;
        const float4 *p = mine + i * 2 * kMaxTeam, a = p[0], b = p[kMaxTeam];
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
        return true;
    }
};
constexpr size_t kHeldGroup = kMaxTeam * 8 * 4;  // bytes of a block's group

template <typename XT, bool VEC, bool DROP>
__global__ void __launch_bounds__(kMaxTeam) layernorm_wide_kernel(const __grid_constant__ LayerNormOp op, int held_groups) {
    extern __shared__ __align__(16) uint8_t ring_smem[];
    __shared__ float2 s[3][32];
    constexpr int team = kMaxTeam;
    const int t = int(threadIdx.x);
    const int64_t row = blockIdx.x;
    const int64_t groups = (op.cols + 8 * team - 1) / (8 * team);
    const Held held(ring_smem, held_groups);
    grid_launch_dependents();
    grid_dependency_wait();
    DropRow k{};
    if constexpr (DROP) k = drop_row(op.drop, drop_offset(op.drop), uint32_t(row));
    float h[8], y[8];
    // h of group i (zero past the row).
    const auto load = [&](int64_t i) {
        if (!held.get(i, h)) load_sum<XT, VEC, DROP>(op, k, row, Cols<VEC>(i, t, team, op.cols), h);
    };
    float sum = 0.f, unused = 0.f;
#pragma unroll 2
    for (int64_t i = 0; i < groups; ++i) {
        load_sum<XT, VEC, DROP>(op, k, row, Cols<VEC>(i, t, team, op.cols), h);
        held.put(i, h);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += h[j];
    }
    block_sum(sum, unused, s[0]);
    const float mean = sum / float(op.cols);
    float d = 0.f, dd = 0.f;
    for (int64_t i = 0; i < groups; ++i) {
        const Cols<VEC> c(i, t, team, op.cols);
        load(i);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float e = j < c.n ? h[j] - mean : 0.f;
            d += e;
            dd += e * e;
        }
    }
    block_sum(d, dd, s[1]);
    const Stats st = stats_of(mean, d, dd, 1.f / float(op.cols), op.eps);
    if (t == 0) {
        if (op.mean) op.mean[row] = st.mean + st.off;
        if (op.rstd) op.rstd[row] = st.rstd;
    }
    float inv = 1.f;
    if (op.mode == TPGEMM_SCALE_ROW) {
        uint32_t amax = 0;
        for (int64_t i = 0; i < groups; ++i) {
            const Cols<VEC> c(i, t, team, op.cols);
            load(i);
            normalise<XT, VEC>(op, st, c, h, y);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < c.n) amax = max(amax, abs_bits(y[j]));
        }
        team_sum_max<false>(unused, amax, s[2]);
        const float scale = row_scale(amax, op.y);
        if (t == 0) op.scale[row] = scale;
        inv = 1.f / scale;
    }
    for (int64_t i = 0; i < groups; ++i) {
        const Cols<VEC> c(i, t, team, op.cols);
        load(i);
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
//
// Aligned rows, read ahead as by the norm. With more than 16 columns to a thread
// what a reduction leaves to be used, w and n, is computed a second time from shared
// memory in place of held in registers, which the columns' sums take. A block's
// teams add up their sums in order at the end.
// Whole rows of at most 16 columns to a thread hold gamma as 32-bit values, which saves
// taking it apart in every row: 8192 x 4096 bf16 with dh 46 us, 50 held as bf16; 8192 x
// 8192 120 and 121, 65536 x 512 60 and 59. With more columns or an index computed in the
// row it takes registers that the rows need: 2048 x 16384 100 and 94, 4096 x 4099 122
// and 108.
template <typename XT, int P, int T, int ROWS>
constexpr bool kWideGamma = ROWS == kWhole && T != 0 && P * kPairs<XT> <= 8;

template <typename XT, int P, int T, int ROWS, bool DROP>
__global__ void __launch_bounds__(RowKernel<P, T, true>::kThreads, RowKernel<P, T, true>::kBlocks)
    layernorm_grad_rows_kernel(const __grid_constant__ LayerNormGradOp op, const RingPlan plan) {
    constexpr int N = kPairs<XT>;
    extern __shared__ __align__(16) uint8_t ring_smem[];
    __shared__ float2 s[2][32];
    __shared__ float stats[kMaxDepth][16][2];  // mean and rstd of the rows ahead, for each warp
    constexpr bool kAgain = P * N > 8;
    const Team<T> team(plan.team);
    const int teams = int(blockDim.x) / team.threads();
    const int64_t stride = int64_t(gridDim.x) * teams;
    int64_t row = int64_t(blockIdx.x) * teams + team.index;
    const int cols = int(op.cols), depth = plan.depth;
    const bool rows_wanted = op.dX || op.dR, add_dh = rows_wanted && op.dH;
    const Ring<XT, P, RowKernel<P, T, true>::kThreads, ROWS> ring(ring_smem, depth, add_dh ? 3 : 2);
    const Weights<XT, P, ROWS, kWideGamma<XT, P, T, ROWS>> weights{
        plan.weights_at ? reinterpret_cast<uint4*>(ring_smem + plan.weights_at) + team.t : nullptr, op.g, team.threads(), cols};
    const auto column = [&](int i) { return kCols<XT> * (i * team.threads() + team.t); };
    // Whether piece i is in the row (of rows anywhere: the warp's first lane's is), and its columns there.
    const auto has = [&](int i) {
        return ROWS == kWhole || column(i) - (ROWS == kAnywhere ? kCols<XT> * int(threadIdx.x & 31) : 0) < cols;
    };
    const auto count = [&](int i) { return ROWS == kAnywhere ? max(0, min(kCols<XT>, cols - column(i))) : kCols<XT>; };
    // (first: whether r may be one of the first eight rows, a constant. Blocks' later rows
    // are not: a turn of the grid takes all rows, or 152 and more.)
    const auto fetch = [&](int64_t r, int slot, auto first) {
        constexpr bool kFirst = decltype(first)::value;
        uint4* const place = ring.row(slot);
        if (r < op.rows) {
            // (A load that the next row waits for would take as long as that row.)
            const int lane = threadIdx.x & 31;
            if (lane < 2)
                cp_async_4(smem_u32(&stats[slot][threadIdx.x >> 5][lane]), (lane ? op.rstd : op.mean) + r);
            const XT* dy = static_cast<const XT*>(op.dY) + r * op.lddy;
            const XT* h = static_cast<const XT*>(op.H) + r * op.ldh;
            const XT* dh = static_cast<const XT*>(op.dH) + (add_dh ? r * op.lddh : 0);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                if (!has(i)) continue;
                ring.template fetch<kFirst>(place, 0, i, op.dY, dy, column(i), cols);
                ring.template fetch<kFirst>(place, 1, i, op.H, h, column(i), cols);
                if (add_dh) ring.template fetch<kFirst>(place, 2, i, op.dH, dh, column(i), cols);
            }
        }
        cp_async_commit();
    };
    grid_launch_dependents();
    grid_dependency_wait();
    if (ROWS == kAnywhere) fetch(row, 0, std::true_type());
    for (int i = ROWS == kAnywhere; i < depth; ++i) fetch(row + i * stride, i, std::false_type());
    if (rows_wanted && weights.mine) {
        if (team.index == 0)
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (has(i)) weights.hold(0, i, op.gamma, column(i));
        if (teams > 1) __syncthreads();  // (else each thread reads its own)
    }
    DropOffset offset{};
    if constexpr (DROP) offset = drop_offset(op.drop);
    const float inv_n = 1.f / float(op.cols);
    F2 ag[P][N], ab[P][N];
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) ag[i][j] = ab[i][j] = f2(0.f);
    for (int slot = 0, turn = 0; row < op.rows; row += stride, turn ^= 1, slot = slot + 1 == depth ? 0 : slot + 1) {
        ring.wait();
        __syncwarp();
        const float mean = stats[slot][threadIdx.x >> 5][0], rstd = stats[slot][threadIdx.x >> 5][1];
        uint4* const place = ring.row(slot);
        F2 kept_w[kAgain ? 1 : P][N], kept_n[kAgain ? 1 : P][N];
        const int off_dy = off16(static_cast<const XT*>(op.dY) + row * op.lddy);
        const int off_h = off16(static_cast<const XT*>(op.H) + row * op.ldh);
        const int off_dh = add_dh ? off16(static_cast<const XT*>(op.dH) + row * op.lddh) : 0;
        // dY and (H - mean) rstd of piece i.
        const auto load = [&](int i, F2 (&w)[N], F2 (&n)[N]) {
            ring.get(place, 0, i, off_dy, w);
            ring.get(place, 1, i, off_h, n);
#pragma unroll
            for (int j = 0; j < N; ++j) n[j] = mul(add(n[j], f2(-mean)), f2(rstd));
        };
        const auto times_gamma = [&](int i, F2 (&w)[N]) {
            F2 g[N];
            weights.get(0, i, op.gamma, column(i), g);
#pragma unroll
            for (int j = 0; j < N; ++j) w[j] = mul(w[j], g[j]);
        };
        F2 pw[N], pn[N];
        zero(pw);
        zero(pn);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (!has(i)) continue;
            F2 (&w)[N] = kept_w[kAgain ? 0 : i], (&n)[N] = kept_n[kAgain ? 0 : i];
            load(i, w, n);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                ag[i][j] = fma(w[j], n[j], ag[i][j]);
                ab[i][j] = add(ab[i][j], w[j]);
            }
            if (rows_wanted) {
                times_gamma(i, w);
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    pw[j] = add(pw[j], w[j]);
                    pn[j] = fma(w[j], n[j], pn[j]);
                }
            }
        }
        if (rows_wanted) {
            float both[2] = {sum_of(pw), sum_of(pn)};
            team.sum(both, s[turn]);
            const F2 sw = f2(-both[0] * inv_n), swn = f2(-both[1] * inv_n);
            DropRow words{};
            if constexpr (DROP) words = drop_row(op.drop, offset, uint32_t(row));
#pragma unroll
            for (int i = 0; i < P; ++i) {
                if (!has(i)) continue;
                F2 (&w)[N] = kept_w[kAgain ? 0 : i], (&n)[N] = kept_n[kAgain ? 0 : i];
                if constexpr (kAgain) {
                    load(i, w, n);
                    times_gamma(i, w);
                }
                F2 dt[N];
                zero(dt);
                if (add_dh) ring.get(place, 2, i, off_dh, dt);
#pragma unroll
                for (int j = 0; j < N; ++j) dt[j] = fma(fma(n[j], swn, add(w[j], sw)), f2(rstd), dt[j]);
                if (op.dR) store_piece<ROWS>(static_cast<XT*>(op.dR) + row * op.lddr + column(i), count(i), dt);
                if (op.dX) {
                    if constexpr (DROP) {
                        keep_pairs(op.drop, words, column(i), dt);
#pragma unroll
                        for (int j = 0; j < N; ++j) dt[j] = mul(dt[j], f2(op.drop.scale));
                    }
                    store_piece<ROWS>(static_cast<XT*>(op.dX) + row * op.lddx + column(i), count(i), dt);
                }
            }
        }
        __syncwarp();  // (the warp has read its statistics)
        fetch(row + depth * stride, slot, std::false_type());
    }
    cp_async_wait<0>();
    if (!op.partial) return;
    float* out = op.partial + int64_t(blockIdx.x) * 2 * op.cols;
    if (teams == 1) {
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (has(i)) {
                store_piece<ROWS>(out + column(i), count(i), ag[i]);
                store_piece<ROWS>(out + op.cols + column(i), count(i), ab[i]);
            }
        return;
    }
    // Through the ring's place, where nothing is on its way: gamma's sums, then beta's.
    float* const sums = reinterpret_cast<float*>(ring_smem);  // [teams][padded columns]
    const int pitch = kCols<XT> * P * team.threads();
    const auto join = [&](const F2 (&a)[P][N], float* to) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < P; ++i) store_pairs(sums + team.index * pitch + column(i), a[i]);
        __syncthreads();
        for (int c = int(threadIdx.x); c < cols; c += int(blockDim.x)) {
            float v = 0.f;
            for (int r = 0; r < teams; ++r) v += sums[r * pitch + c];
            to[c] = v;
        }
    };
    join(ag, out);
    join(ab, out + op.cols);
}

// Wider rows: dt a row to a block, w and n of the first `held` groups (24576 columns)
// kept in shared memory, and the column sums apart (2048 x 20480 bf16 with dropout and
// dh 191 us, 344 with all read again, element by element).
template <typename XT, bool VEC, bool DROP>
__global__ void __launch_bounds__(kMaxTeam) layernorm_grad_wide_kernel(const __grid_constant__ LayerNormGradOp op,
                                                                       int held_groups) {
    extern __shared__ __align__(16) uint8_t ring_smem[];
    __shared__ float2 s[32];
    constexpr int team = kMaxTeam;
    const int t = int(threadIdx.x);
    const int64_t row = blockIdx.x;
    const int64_t groups = (op.cols + 8 * team - 1) / (8 * team);
    const Held held(ring_smem, 2 * held_groups);
    grid_launch_dependents();
    grid_dependency_wait();
    DropRow k{};
    if constexpr (DROP) k = drop_row(op.drop, drop_offset(op.drop), uint32_t(row));
    const float rstd = op.rstd[row], mean = op.mean[row];
    float w[8], n[8];
    const auto load = [&](int64_t i, const Cols<VEC>& c) {
        float g[8];
        load_cols<XT, VEC>(op.dY, row * op.lddy, c, w);
        load_cols<XT, VEC>(op.H, row * op.ldh, c, n);
        load_gamma<XT, VEC>(op.gamma, op.g, c, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[j] *= g[j];  // (0 past the row)
            n[j] = (n[j] - mean) * rstd;
        }
    };
    float sw = 0.f, swn = 0.f;
    for (int64_t i = 0; i < groups; ++i) {
        load(i, Cols<VEC>(i, t, team, op.cols));
        held.put(2 * i, w);
        held.put(2 * i + 1, n);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            sw += w[j];
            swn += w[j] * n[j];
        }
    }
    block_sum(sw, swn, s);
    sw /= float(op.cols);
    swn /= float(op.cols);
    for (int64_t i = 0; i < groups; ++i) {
        const Cols<VEC> c(i, t, team, op.cols);
        float dt[8];
        if (op.dH) {
            load_cols<XT, VEC>(op.dH, row * op.lddh, c, dt);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) dt[j] = 0.f;
        }
        if (held.get(2 * i, w)) held.get(2 * i + 1, n);
        else load(i, c);
#pragma unroll
        for (int j = 0; j < 8; ++j) dt[j] += rstd * (w[j] - sw - n[j] * swn);
        if (op.dR) store_cols<XT, VEC>(op.dR, row * op.lddr, c, dt);
        if (op.dX) {
            if constexpr (DROP) {
                keep_cols<VEC>(op.drop, k, c, dt);
#pragma unroll
                for (int j = 0; j < 8; ++j) dt[j] *= op.drop.scale;
            }
            store_cols<XT, VEC>(op.dX, row * op.lddx, c, dt);
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
#pragma unroll 8
    for (int64_t r = begin; r < end; ++r) {
        const float dy = to_f32(static_cast<const XT*>(op.dY)[r * op.lddy + c]);
        g += dy * ((to_f32(static_cast<const XT*>(op.H)[r * op.ldh + c]) - op.mean[r]) * op.rstd[r]);
        b += dy;
    }
    float* out = op.partial + int64_t(blockIdx.y) * 2 * op.cols + c;
    out[0] = g;
    out[op.cols] = b;
}

// Rows of up to kMaxHeld columns. A reduction costs each warp that takes
// part as many instructions as 16 columns, so the norm has four pieces to a thread,
// its gradients 16 columns; fewer of rows that a warp then holds whole; twice as many
// of rows wider than 512 such threads; and of few rows one, for the shortest time to
// the end.
constexpr int most_pieces(int elem, bool grad) { return grad && elem != TPGEMM_ELEM_F32 ? 2 : 4; }

struct RowSpread {
    int p, t;         // the kernel's P and T
    bool whole;       // all of the team's pieces are in the row
    int team, teams;  // threads of a team, teams of a block
    int blocks;       // to an SM
    int threads() const { return team * teams; }
};
RowSpread row_spread(int64_t rows, int64_t cols, int elem, bool grad, bool aligned) {
    const int pieces = int((cols * elem_size(elem) + 15) / 16);
    const int most = rows <= kSms ? 1 : most_pieces(elem, grad);
    int p = 1;
    while (p < most && 32 * p < pieces) p *= 2;
    while (512 * p < pieces) p *= 2;
    const int team = (pieces + 32 * p - 1) / (32 * p) * 32;
    const bool whole = aligned && most > 1 && team * p == pieces;
    const int t = whole && (team & (team - 1)) == 0 ? team : 0;
    const int threads = t == 0 ? any_threads(p, grad) : grad && t <= 256 ? 256 : 512;
    const int teams = int(std::max<int64_t>(1, std::min<int64_t>(threads / team, rows / kSms)));
    return {p, t, whole, team, teams, std::max(1, std::min((t == 0 ? threads : grad ? 512 : 1024) / (team * teams), 8))};
}

constexpr int kRingBytes = 216 * 1024;  // of an SM, for its blocks
// `step`: threads that a block's places are laid out for. Of a team's only row no other
// is copied ahead, and the weights, which it reads once, are held where it is the
// block's only team: they come beside the row and not after its reductions.
RingPlan ring_plan(RowSpread* s, bool anywhere, int64_t rows, int step, int inputs, int elem, int vectors, int vector_elem,
                   size_t* bytes) {
    const size_t row = size_t(inputs) * s->p * (step + (anywhere ? step / 32 : 0)) * 16;  // of all teams
    const int64_t turns = (rows + int64_t(kSms) * s->blocks * s->teams - 1) / (int64_t(kSms) * s->blocks * s->teams);
    size_t held = turns == 1 && s->teams > 1 ? 0 : size_t(vectors) * s->p * s->team * 16 * elem_size(vector_elem) / elem_size(elem);
    while (s->blocks > 1 && held + row > size_t(kRingBytes / s->blocks)) --s->blocks;
    const size_t have = size_t(kRingBytes / s->blocks);
    if (held + row > have) held = 0;
    const int fit = int((have - held) / row);
    const int depth = int(std::max<int64_t>(1, std::min<int64_t>(turns, std::min(kMaxDepth, fit))));
    *bytes = depth * row + held;
    return {s->team, depth, held ? int(depth * row) : 0};
}

// f(P, T, ROWS) of the spread's kernel, as integral constants. MOST: most_pieces;
// TWICE: whether rows of up to kMaxHeld columns come to more than MOST.
template <int MOST, bool TWICE, typename F>
cudaError_t with_spread(const RowSpread& s, bool aligned, F&& f) {
    using std::integral_constant;
    const auto pieces = [&](auto g) {
        if constexpr (TWICE)
            if (s.p == 2 * MOST) return g(integral_constant<int, 2 * MOST>());
        if constexpr (MOST == 4)
            if (s.p == 4) return g(integral_constant<int, 4>());
        return s.p == 2 ? g(integral_constant<int, 2>()) : g(integral_constant<int, 1>());
    };
    constexpr integral_constant<int, 0> any{};
    constexpr integral_constant<int, MOST> most{};
    if (s.t == 0 && !s.whole)
        return pieces([&](auto p) {
            return aligned ? f(p, any, integral_constant<int, kAligned>()) : f(p, any, integral_constant<int, kAnywhere>());
        });
    constexpr integral_constant<int, kWhole> whole{};
    constexpr integral_constant<int, 512> t512{};
    if (s.t == 0) {  // (a team of 96 threads or more, with as many pieces as MOST at least)
        if constexpr (TWICE)
            if (s.p > MOST) return f(integral_constant<int, 2 * MOST>(), any, whole);
        return f(most, any, whole);
    }
    if (s.t == 32) {  // (as many pieces as MOST at the most)
        constexpr integral_constant<int, 32> t32{};
        if constexpr (MOST == 4)
            if (s.p == 4) return f(integral_constant<int, 4>(), t32, whole);
        return s.p == 2 ? f(integral_constant<int, 2>(), t32, whole) : f(integral_constant<int, 1>(), t32, whole);
    }
    if constexpr (TWICE)
        if (s.p > MOST) return f(integral_constant<int, 2 * MOST>(), t512, whole);
    switch (s.t) {
        case 64: return f(most, integral_constant<int, 64>(), whole);
        case 128: return f(most, integral_constant<int, 128>(), whole);
        case 256: return f(most, integral_constant<int, 256>(), whole);
        default: return f(most, t512, whole);
    }
}

// Lets a kernel use all of kRingBytes: the most that any call of it wants, and not this
// call's, since the limit is the kernel's and another thread may be about to launch it.
template <typename F>
cudaError_t allow_ring(F fn) {
    return cudaFuncSetAttribute(reinterpret_cast<const void*>(fn), cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
}

template <typename F, typename Op>
cudaError_t launch_ring(F fn, int64_t blocks, int threads, size_t bytes, const RingPlan& plan, cudaStream_t stream,
                        const Op& op) {
    if (bytes > 40 * 1024) {  // (with the kernel's own, more than a block has without asking)
        const cudaError_t e = allow_ring(fn);
        if (e != cudaSuccess) return e;
    }
    return launch_dependent(fn, dim3(unsigned(blocks)), dim3(unsigned(threads)), bytes, stream, op, plan);
}

// A block to a row, with room for `values` values of as many columns as fit.
template <typename F, typename Op>
cudaError_t launch_wide(F fn, const Op& op, int values, cudaStream_t stream) {
    const int64_t groups = (op.cols + 8 * kMaxTeam - 1) / (8 * kMaxTeam);
    const int held = int(std::min<int64_t>(groups, int64_t(kRingBytes / kHeldGroup) / values));
    const size_t bytes = size_t(held) * values * kHeldGroup;
    const cudaError_t e = allow_ring(fn);
    if (e != cudaSuccess) return e;
    return launch_dependent(fn, dim3(unsigned(op.rows)), dim3(kMaxTeam), bytes, stream, op, held);
}

template <typename XT, bool DROP>
cudaError_t launch_norm(const LayerNormOp& op, bool aligned, cudaStream_t stream) {
    if (op.rows > 0x7fffffff) return cudaErrorInvalidValue;
    if (op.cols > kMaxHeld)
        return launch_wide(aligned && op.cols % 8 == 0 ? layernorm_wide_kernel<XT, true, DROP>
                                                       : layernorm_wide_kernel<XT, false, DROP>, op, 1, stream);
    RowSpread s = row_spread(op.rows, op.cols, op.x, false, aligned);
    return with_spread<4, sizeof(XT) == 4>(s, aligned, [&](auto p, auto t, auto where) {
        constexpr int P = decltype(p)::value, T = decltype(t)::value;
        size_t bytes;
        const RingPlan plan = ring_plan(&s, !aligned, op.rows, RowKernel<P, T, false>::kThreads, op.R ? 2 : 1, op.x,
                                        op.beta ? 2 : 1, op.g, &bytes);
        const int64_t blocks = std::min<int64_t>((op.rows + s.teams - 1) / s.teams, int64_t(kSms) * s.blocks);
        return launch_ring(layernorm_rows_kernel<XT, P, T, decltype(where)::value, DROP>, blocks, s.threads(), bytes,
                           plan, stream, op);
    });
}

template <typename XT>
cudaError_t launch_norm_typed(const LayerNormOp& op, cudaStream_t stream) {
    // (The kernel of wider rows stores eight columns at a time.)
    const int y_bytes = (op.cols > kMaxHeld ? 8 : kCols<XT>) * elem_size(op.y);
    const bool aligned = op.cols % kCols<XT> == 0 && rows_aligned(op.X, op.ldx, op.rows, op.x, 16) &&
                         rows_aligned(op.R, op.ldr, op.rows, op.x, 16) &&
                         rows_aligned(op.H, op.ldh, op.rows, op.x, 16) &&
                         rows_aligned(op.Y, op.ldy, op.rows, op.y, std::min(16, y_bytes)) &&
                         rows_aligned(op.gamma, 0, 1, op.g, 16) && rows_aligned(op.beta, 0, 1, op.g, 16);
    return op.drop.on ? launch_norm<XT, true>(op, aligned, stream) : launch_norm<XT, false>(op, aligned, stream);
}

// What the SMs hold, and no more than there are rows.
int grad_row_blocks(int64_t rows, const RowSpread& s) {
    const int64_t most = (rows + s.teams - 1) / s.teams;
    return int(std::min<int64_t>(most, int64_t(kSms) * s.blocks));
}

int wide_strips(int64_t rows) {
    const int64_t most = (rows + 15) / 16;
    return int(most < 1 ? 1 : (most < 64 ? most : 64));
}

template <typename XT, bool DROP>
cudaError_t launch_grad(const LayerNormGradOp& op, bool aligned, int* strips, cudaStream_t stream) {
    RowSpread s = row_spread(op.rows, op.cols, op.x, true, aligned);
    return with_spread<sizeof(XT) == 4 ? 4 : 2, true>(s, aligned, [&](auto p, auto t, auto where) {
        constexpr int P = decltype(p)::value, T = decltype(t)::value;
        size_t bytes;
        const RingPlan plan = ring_plan(&s, !aligned, op.rows, RowKernel<P, T, true>::kThreads,
                                        op.dH && (op.dX || op.dR) ? 3 : 2, op.x, 1,
                                        kWideGamma<XT, P, T, decltype(where)::value> ? TPGEMM_ELEM_F32 : int(op.g), &bytes);
        if (s.teams > 1) bytes = std::max(bytes, size_t(P) * kCols<XT> * s.threads() * 4);  // (the teams' sums)
        *strips = grad_row_blocks(op.rows, s);
        return launch_ring(layernorm_grad_rows_kernel<XT, P, T, decltype(where)::value, DROP>, *strips, s.threads(),
                           bytes, plan, stream, op);
    });
}

template <typename XT>
cudaError_t launch_grad_typed(const LayerNormGradOp& op, cudaStream_t stream) {
    int strips = wide_strips(op.rows);
    const bool drop = op.drop.on != 0;
    const bool aligned = op.cols % kCols<XT> == 0 && rows_aligned(op.dY, op.lddy, op.rows, op.x, 16) &&
                         rows_aligned(op.H, op.ldh, op.rows, op.x, 16) &&
                         rows_aligned(op.dH, op.lddh, op.rows, op.x, 16) &&
                         rows_aligned(op.dX, op.lddx, op.rows, op.x, 16) &&
                         rows_aligned(op.dR, op.lddr, op.rows, op.x, 16) &&
                         rows_aligned(op.gamma, 0, 1, op.g, 16);
    cudaError_t e = cudaSuccess;
    if (op.cols > kMaxHeld) {
        // The columns first: dX or dR may be written over dY or H.
        if (op.partial) {
            const dim3 grid(unsigned((op.cols + 255) / 256), static_cast<unsigned>(strips));
            e = launch_dependent(layernorm_columns_kernel<XT>, grid, dim3(256), 0, stream, op, strips);
        }
        if (e == cudaSuccess && (op.dX || op.dR)) {
            auto fn = aligned && op.cols % 8 == 0
                          ? (drop ? layernorm_grad_wide_kernel<XT, true, true> : layernorm_grad_wide_kernel<XT, true, false>)
                          : (drop ? layernorm_grad_wide_kernel<XT, false, true> : layernorm_grad_wide_kernel<XT, false, false>);
            e = launch_wide(fn, op, 2, stream);
        }
    } else {
        e = drop ? launch_grad<XT, true>(op, aligned, &strips, stream) : launch_grad<XT, false>(op, aligned, &strips, stream);
    }
    if (e != cudaSuccess || !op.partial) return e;
    return launch_column_sums(op.partial, strips, op.cols, op.dgamma, op.dbeta, op.grad, stream);
}

}  // namespace

template <typename XT>
cudaError_t layernorm_of(const LayerNormOp& op, cudaStream_t stream) {
    return launch_norm_typed<XT>(op, stream);
}

template <typename XT>
cudaError_t layernorm_grad_of(const LayerNormGradOp& op, cudaStream_t stream) {
    return launch_grad_typed<XT>(op, stream);
}

}  // namespace tpg
