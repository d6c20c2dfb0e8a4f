// Rows of the norms: how a row's columns are spread over the threads that share
// it (a team: a warp for narrow rows, else a block), their accesses, and the
// team's reductions.
#pragma once

#include <type_traits>

#include "ptx.cuh"
#include "vec8.cuh"

namespace tpg {
namespace {

constexpr int kMaxTeam = 1024;               // threads of a row
constexpr int kMaxHeld = kMaxTeam * 8 * 2;   // columns a team holds in registers
constexpr int kWarpRows = 8;                 // rows of a block when a row is a warp's

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Scale of a row whose largest |value| has the given 32-bit pattern. Maxima are
// taken of the patterns, so that infinities and NaN (the largest ones) are kept.
__device__ __forceinline__ float row_scale(uint32_t amax, int elem) {
    const float top = elem == TPGEMM_ELEM_E4M3 ? 448.f : 57344.f;
    if (amax >= 0x7f800000u) return __uint_as_float(0x7fffffffu);
    return fmaxf(__uint_as_float(amax) / top, 1.17549435e-38f);
}

// A thread's eight columns of group i of a row that `team` threads share:
// neighbouring ones when rows are aligned, else team columns apart, so that
// either way a warp's accesses are contiguous.
template <bool VEC>
struct Cols {
    int64_t first;  // of the eight
    int step, n;    // distance between them, and how many lie in the row
    __device__ __forceinline__ Cols(int64_t i, int t, int team, int64_t cols) {
        const int64_t base = i * 8 * team;
        first = VEC ? base + 8 * t : base + t;
        step = VEC ? 1 : team;
        const int64_t left = cols - first;
        n = left <= 0 ? 0 : VEC ? (left < 8 ? int(left) : 8)
                                : int(min(int64_t(8), (left + team - 1) / team));
    }
};

template <typename T, bool VEC>
__device__ __forceinline__ void load_cols(const void* base, int64_t row, const Cols<VEC>& c,
                                          float (&f)[8]) {
    if constexpr (VEC) {
        // (Aligned rows are whole groups of eight.)
        if (c.n == 8) {
            load8<T>(base, row + c.first, true, 8, f);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = 0.f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            f[j] = j < c.n ? to_f32(static_cast<const T*>(base)[row + c.first + int64_t(j) * c.step]) : 0.f;
    }
}

// A group as it is loaded ahead of its use: 16-bit elements stay packed.
template <typename T, bool VEC>
struct Ahead {
    static constexpr bool kPacked = VEC && sizeof(T) == 2;
    uint4 raw;
    float f[kPacked ? 1 : 8];
    __device__ __forceinline__ void load(const void* base, int64_t row, const Cols<VEC>& c) {
        if constexpr (kPacked) {
            raw = make_uint4(0, 0, 0, 0);
            if (c.n == 8) raw = *reinterpret_cast<const uint4*>(static_cast<const T*>(base) + row + c.first);
        } else {
            load_cols<T, VEC>(base, row, c, f);
        }
    }
    __device__ __forceinline__ void get(float (&out)[8]) const {
        if constexpr (kPacked) {
            unpack8<T>(raw, out);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) out[j] = f[j];
        }
    }
};

template <typename T, bool VEC>
__device__ __forceinline__ void store_cols(void* base, int64_t row, const Cols<VEC>& c,
                                           const float (&f)[8]) {
    if constexpr (VEC) {
        if (c.n == 8) {
            if constexpr (sizeof(T) == 1)
                *reinterpret_cast<uint2*>(static_cast<T*>(base) + row + c.first) =
                    pack8_fp8(f, std::is_same<T, e4m3>::value ? __NV_E4M3 : __NV_E5M2);
            else
                store8<T>(base, row + c.first, true, 8, f);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < c.n)
                static_cast<T*>(base)[row + c.first + int64_t(j) * c.step] = from_f32<T>(f[j]);
    }
}

template <typename XT, bool VEC>
__device__ __forceinline__ void load_gamma(const void* gamma, int elem, const Cols<VEC>& c,
                                           float (&f)[8]) {
    if (elem == TPGEMM_ELEM_F32)
        load_cols<float, VEC>(gamma, 0, c, f);
    else
        load_cols<XT, VEC>(gamma, 0, c, f);
}

// Sum of a and maximum of b over a warp, or over the block through `s`.
template <bool WARP>
__device__ __forceinline__ void team_sum_max(float& a, uint32_t& b, float2* s) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    b = __reduce_max_sync(0xffffffffu, b);
    if constexpr (!WARP) {
        const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
        if (lane == 0) s[threadIdx.x >> 5] = make_float2(a, __uint_as_float(b));
        __syncthreads();
        const float2 v = lane < nw ? s[lane] : make_float2(0.f, 0.f);
        a = v.x;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
        b = __reduce_max_sync(0xffffffffu, __float_as_uint(v.y));
    }
}

// Maximum over a warp, or over the block through an `s` that it may still read.
template <bool WARP>
__device__ __forceinline__ void team_max(uint32_t& b, float2* s) {
    b = __reduce_max_sync(0xffffffffu, b);
    if constexpr (!WARP) {
        const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
        __syncthreads();
        if (lane == 0) s[threadIdx.x >> 5].y = __uint_as_float(b);
        __syncthreads();
        b = __reduce_max_sync(0xffffffffu, lane < nw ? __float_as_uint(s[lane].y) : 0u);
    }
}

// How a row is spread: threads of a team (a warp's rows come kWarpRows to a
// block), groups of eight columns to a thread (0: wider than the registers).
struct Spread {
    int team, v;
    bool warp;
    int threads() const { return warp ? 32 * kWarpRows : team; }
    int rows() const { return warp ? kWarpRows : 1; }
};

inline bool rows_aligned(const void* p, int64_t ld, int64_t rows, int elem, int bytes) {
    return !p || (reinterpret_cast<uintptr_t>(p) % bytes == 0 &&
                  (rows <= 1 || (ld * elem_size(elem)) % bytes == 0));
}

}  // namespace
}  // namespace tpg
