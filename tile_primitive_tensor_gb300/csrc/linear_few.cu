// The linear layer for few tokens (M <= 16): every weight is read once and used
// for at most 16 rows of A, so the weights' way from memory is what counts.
//
// No shared-memory staging: warp-level mma.sync takes 16 rows of W as its A
// operand and 8 or 16 tokens as its B operand, and each thread loads 16 bytes
// of neighbouring K straight into its fragments. The order of K within a product
// does not matter as long as both operands agree on it, so the four threads of a
// row simply hold 16 bytes each: with 16-bit elements e0..e7, the first
// m16n8k16 takes (e0 e1), (e2 e3) as its two K pairs, the second (e4 e5),
// (e6 e7); W and A are loaded alike. 8-bit elements are widened to f16, which
// holds every e4m3 and e5m2 value.
//
// A block takes 16 rows of W, its 8 warps alternate runs of K; with few rows a
// cluster of blocks shares them. Partial sums meet in shared memory and are
// added in a fixed order. Bound by memory: the weights' bytes, and for few of
// them by its latency (one token of 4096 x 4096 bf16: 8.5 us, of which 4.9 are
// the bytes; unaligned rows, 12 x 4096 x 4097: 33 us, 42 element by element).
#include <algorithm>

#include "launch.cuh"
#include "ptx.cuh"
#include "vec8.cuh"

namespace tpg {
namespace {

constexpr int kWarps = 8;
constexpr int kRows = 16;   // rows of W in a block (gated: 8 of each half)
constexpr int kRun = 4;     // 16-byte loads of a row that a thread has in flight at a time
constexpr int kPrefetch = 2;  // runs of a warp asked for ahead
constexpr int64_t kManyRows = 2 * kSms * kRows;  // of W: more than two blocks to an SM

// The 16 bytes of row r from element k on (zero past K or for no row).
// (A coherent load: the weights may be what the previous grid, which this one
// starts beside, still writes until the dependency is waited for.)
template <typename T>
__device__ __forceinline__ uint4 load16(const T* r, bool live, int64_t k, int64_t K) {
    constexpr int E = 16 / sizeof(T);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (!live || k >= K) return v;
    if (k + E <= K) {
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(r + k));
        return v;
    }
    using Raw = typename std::conditional<sizeof(T) == 1, uint8_t, uint16_t>::type;
    const Raw* p = reinterpret_cast<const Raw*>(r);
    uint32_t w[4] = {};
#pragma unroll
    for (int i = 0; i < E; ++i)
        if (k + i < K) w[i * sizeof(T) / 4] |= uint32_t(p[k + i]) << (8 * (i * sizeof(T) % 4));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// Two neighbouring 8-bit elements as an f16 pair.
template <typename T>
__device__ __forceinline__ uint32_t widen(uint32_t two) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        __nv_fp8x2_storage_t(two), std::is_same<T, e4m3>::value ? __NV_E4M3 : __NV_E5M2);
    return uint32_t(h.x) | (uint32_t(h.y) << 16);
}

// acc += the product of 16 rows of W (lo: rows 0..7, hi: rows 8..15) and the
// tokens of x over these 16 bytes of K.
template <typename T>
__device__ __forceinline__ void multiply(float (&acc)[4], const uint4& lo, const uint4& hi,
                                         const uint4& x) {
    const uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, h[4] = {hi.x, hi.y, hi.z, hi.w},
                   t[4] = {x.x, x.y, x.z, x.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const uint32_t a[4] = {l[i], h[i], l[i + 1], h[i + 1]};
            mma_m16n8k16<std::is_same<T, __nv_bfloat16>::value>(acc, a, t[i], t[i + 1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t a[4] = {widen<T>(l[i] & 0xffffu), widen<T>(h[i] & 0xffffu),
                                   widen<T>(l[i] >> 16), widen<T>(h[i] >> 16)};
            mma_m16n8k16<false>(acc, a, widen<T>(t[i] & 0xffffu), widen<T>(t[i] >> 16));
        }
    }
}

// TT: token tiles of 8.
template <typename T, typename O, int TT, bool VEC>
__global__ void __launch_bounds__(32 * kWarps) linear_few_kernel(const __grid_constant__ LinearOp op,
                                                                 int split) {
    __shared__ float part[kWarps][8 * TT][kRows + 1];
    __shared__ float mine[8 * TT][kRows];
    constexpr int E = 16 / sizeof(T);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int rank = int(cluster_ctarank());
    // (More than 16 rows of A, 16 to a group of blocks, only come with K = 0.)
    const int per = op.gated ? kRows / 2 : kRows;  // outputs of a token
    const int64_t tiles = (op.N + per - 1) / per, tile = blockIdx.x / split;
    const int64_t n0 = tile % tiles * per, m0 = tile / tiles * kFewTokens;
    const T* W = static_cast<const T*>(op.b.p);
    const T* A = static_cast<const T*>(op.a.p);
    const bool live_lo = n0 + g < op.N, live_hi = op.gated ? live_lo : n0 + g + 8 < op.N;
    const T* lo_row = W + (live_lo ? n0 + g : 0) * op.b.ld;
    const T* hi_row = W + (live_hi ? n0 + g + (op.gated ? op.N : 8) : 0) * op.b.ld;
    const int64_t step = 4 * E * kRun;  // K of one run of a warp
    const int64_t stride = step * kWarps * split;
    grid_launch_dependents();
    // Ask L2 for the first weights before waiting for the previous grid: its
    // writes land in L2 too, so no line there is ever stale.
    if (VEC && (t4 & 1) == 0) {
        for (int j = 0; j < kPrefetch; ++j) {
            const int64_t k = (int64_t(rank) * kWarps + warp) * step + j * stride + t4 * (2 * E * kRun / 2);
            if (k < op.K) {
                if (live_lo) prefetch_l2(lo_row + k);
                if (live_hi) prefetch_l2(hi_row + k);
            }
        }
    }
    grid_dependency_wait();
    float acc[TT][4] = {};
    // Rows that start anywhere are read as the aligned 16 bytes that each lane's
    // start in; a row's four lanes pass them on.
    const auto load_run = [&](const T* row, bool live, int64_t k0, uint4 (&out)[kRun]) {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < kRun; ++i) out[i] = load16<T>(row, live, k0 + (4 * i + t4) * E, op.K);
        } else {
            const uint8_t* bytes = reinterpret_cast<const uint8_t*>(row);
            const int off = int(reinterpret_cast<uintptr_t>(bytes) & 15u);
            const int64_t len = live ? op.K * int64_t(sizeof(T)) : 0, at = k0 * int64_t(sizeof(T)) + 16 * t4 - off;
            Window w[kRun + 1];
#pragma unroll
            for (int i = 0; i < kRun; ++i) w[i] = load_window(bytes, at + 64 * i, len);
            w[kRun] = t4 == 0 ? load_window(bytes, at + 64 * kRun, len) : make_uint4(0, 0, 0, 0);
            const int from = (lane & ~3) | ((t4 + 1) & 3);
            Window here = shuffle_window(w[0], from);
#pragma unroll
            for (int i = 0; i < kRun; ++i) {
                const Window after = shuffle_window(w[i + 1], from);
                out[i] = join_windows(w[i], t4 == 3 ? after : here, off);  // (zero past K)
                here = after;
            }
        }
    };
    for (int64_t k0 = (int64_t(rank) * kWarps + warp) * step; k0 < op.K; k0 += stride) {
        uint4 lo[kRun], hi[kRun], x[TT][kRun];
        load_run(lo_row, live_lo, k0, lo);
        load_run(hi_row, live_hi, k0, hi);
#pragma unroll
        for (int u = 0; u < TT; ++u) {
            const bool live = m0 + 8 * u + g < op.M;
            load_run(A + (live ? m0 + 8 * u + g : 0) * op.a.ld, live, k0, x[u]);
        }
#pragma unroll
        for (int i = 0; i < kRun; ++i)
#pragma unroll
            for (int u = 0; u < TT; ++u) multiply<T>(acc[u], lo[i], hi[i], x[u][i]);
    }
    // acc[u][2 rM + rN]: row g + 8 rM of W, token 8 u + 2 t4 + rN.
#pragma unroll
    for (int u = 0; u < TT; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) part[warp][8 * u + 2 * t4 + (i & 1)][g + 8 * (i >> 1)] = acc[u][i];
    __syncthreads();
    const int row = threadIdx.x % kRows, token = threadIdx.x / kRows;  // 16 tokens' worth of threads
    float v = 0.f;
    if (token < 8 * TT) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += part[w][token][row];
        if (split > 1) mine[token][row] = v;
    }
    if (split > 1) {
        cluster_sync();
        if (token < 8 * TT && token % split == rank) {
            v = 0.f;
            const uint32_t at = smem_u32(&mine[token][row]);
            for (int r = 0; r < split; ++r) {
                float f;
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(mapa_shared(at, uint32_t(r))) : "memory");
                v += f;
            }
        }
    }
    if (op.gated) {  // lanes 8 apart hold an output's gate and factor
        const float u = __shfl_xor_sync(0xffffffffu, v, kRows / 2);
        if (row < kRows / 2 && m0 + token < op.M && token % split == rank && n0 + row < op.N)
            with_act(op.e.act, [&](auto act) {
                epilogue_gated<O, decltype(act)::value>(op.e, op.N, m0 + token, n0 + row, v, u);
            });
    } else if (m0 + token < op.M && token % split == rank && n0 + row < op.N)
        with_act(op.e.act, [&](auto act) {
            epilogue_one<O, decltype(act)::value>(op.e, m0 + token, n0 + row, v);
        });
    if (split > 1) {
        __syncwarp();
        cluster_sync();  // peers have read this block's sums
    }
}

template <typename T, typename O, int TT>
cudaError_t launch_few(const LinearOp& op, int split, cudaStream_t stream) {
    const bool vec = tma_rows(op.a, op.M, op.K, op.dtype) &&
                     tma_rows(op.b, weight_rows(op), op.K, op.dtype);
    auto fn = vec ? linear_few_kernel<T, O, TT, true> : linear_few_kernel<T, O, TT, false>;
    const int64_t blocks = (weight_rows(op) + kRows - 1) / kRows * ((op.M + kFewTokens - 1) / kFewTokens) * split;
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(split);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fn, op, split);
}

template <typename T, typename O>
cudaError_t launch_out(const LinearOp& op, int split, cudaStream_t stream) {
    return op.M <= 8 ? launch_few<T, O, 1>(op, split, stream) : launch_few<T, O, 2>(op, split, stream);
}

template <typename T>
cudaError_t launch_typed(const LinearOp& op, int split, cudaStream_t stream) {
    if (op.e.out == TPGEMM_ELEM_F16) return launch_out<T, __half>(op, split, stream);
    if (op.e.out == TPGEMM_ELEM_BF16) return launch_out<T, __nv_bfloat16>(op, split, stream);
    return launch_out<T, float>(op, split, stream);
}

}  // namespace

bool linear_few_takes(const LinearOp& op) { return op.M <= kFewTokens && !op.a.mn && !op.b.mn; }

// Against the tcgen05 kernels, which stream large weights faster and do not
// widen 8-bit ones, but take 3.5 us at the least. Here a block has 16 weight
// rows whatever their length, so many short rows cost more than few long ones;
// there it is the other way round (one token, N x K, this / tcgen05: 512 x 1024
// bf16 2.5 / 3.6 us, 4096 x 4096 8.5 / 9.7, 1024 x 16384 9.5 / 13.0, 8192 x 2048
// 10.2 / 7.8, 16384 x 512 7.9 / 6.0, 4096 x 8192 15.4 / 14.4; e4m3 4096 x 1024
// 3.8 / 5.0, 1024 x 8192 6.5 / 6.0, 4096 x 4096 8.5 / 7.2).
bool linear_few_wins(const LinearOp& op) {
    const int64_t rows = weight_rows(op);
    if (!tma_rows(op.a, op.M, op.K, op.dtype) || !tma_rows(op.b, rows, op.K, op.dtype)) return true;
    const int64_t weights = rows * op.K * elem_size(op.dtype);
    if (rows > kManyRows && weights > int64_t(4) << 20) return false;
    return weights <= (elem_size(op.dtype) == 1 ? int64_t(6) << 20 : int64_t(40) << 20);
}

cudaError_t launch_linear_few(const LinearOp& op, int sms, cudaStream_t stream) {
    // Clusters share a block's rows of K while that leaves every warp a run of
    // its own and the GPU is not full: 4 blocks of 8 warps to an SM.
    const int64_t tiles = (weight_rows(op) + kRows - 1) / kRows;
    const int64_t run = 4 * (16 / elem_size(op.dtype)) * kRun * kWarps;
    int split = 1;
    while (split < 8 && tiles * split * 2 <= 2 * sms && run * split * 2 <= op.K) split *= 2;
    const int forced = linear_tuning().split;
    if (forced == 1 || forced == 2 || forced == 4 || forced == 8) split = forced;
    switch (op.dtype) {
        case TPGEMM_ELEM_F16: return launch_typed<__half>(op, split, stream);
        case TPGEMM_ELEM_BF16: return launch_typed<__nv_bfloat16>(op, split, stream);
        case TPGEMM_ELEM_E4M3: return launch_typed<e4m3>(op, split, stream);
        default: return launch_typed<e5m2>(op, split, stream);
    }
}

}  // namespace tpg
