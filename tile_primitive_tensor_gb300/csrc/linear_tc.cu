// The linear layer's product on tcgen05: X = P.Q^T with f32 accumulators in
// tensor memory, and the layer's epilogue (scales, bias, activation, residual,
// rounding) on the way out. P's rows run along the tensor-memory lanes and Q's
// along the accumulator's columns; P holds the output's rows (normal) or its
// columns (swapped). Two kernels:
//
//   tile   persistent CTA pairs (tcgen05.mma.cta_group::2, 256 x bn tiles, two
//          accumulators): one tile's epilogue runs under the next one's MMAs.
//   split  one bp x bn tile per cluster of CTAs, each CTA a share of K: for
//          products with too few tiles to fill the GPU. The partial sums are
//          joined through distributed shared memory in rank order, so results
//          repeat, and no global scratch or flag is needed.
//
// Operands are read where they lie, K-contiguous or along their rows, by TMA
// into 128-byte-swizzled stages (K's and the rows' ends read as zero). Every
// wait is bounded: on expiry the kernel records a status, lets its copies and
// MMAs in flight finish, frees tensor memory and returns.
#include <algorithm>
#include <type_traits>

#include "elem.cuh"
#include "linear_tc.h"
#include "ptx.cuh"
#include "tpgemm_internal.h"
#include "vec8.cuh"

namespace tpg {

__device__ int g_linear_status;  // 0 = ok, kStatusTimeout after an expired wait

namespace {

constexpr int kAtom = 8192;  // an operand stored along its rows: 64 K x 64 rows of 16 bits

__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, volatile int* abort,
                                             uint64_t timeout_ns, bool drain = false) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (!drain && *abort) return false;
        if (globaltimer_ns() - t0 > timeout_ns) {
            *abort = 1;
            atomicExch(&g_linear_status, kStatusTimeout);
            return false;
        }
    }
}

// Four MMAs: one 128-byte-wide stage of K. dP / dQ: descriptor templates, the
// stage's operand addresses and the address step of one MMA's K.
template <bool PAIR, bool FP8>
__device__ __forceinline__ void issue_stage(uint32_t acc, uint64_t dP, uint64_t dQ, uint32_t ap,
                                            uint32_t aq, uint32_t step_p, uint32_t step_q,
                                            uint32_t idesc, bool first) {
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
        const uint64_t a = smem_desc_with_addr(dP, ap + kk * step_p);
        const uint64_t b = smem_desc_with_addr(dQ, aq + kk * step_q);
        const uint32_t more = !first || kk != 0;
        if constexpr (PAIR) {
            if constexpr (FP8) tc_mma_f8_pair(acc, a, b, idesc, more);
            else tc_mma_f16_pair(acc, a, b, idesc, more);
        } else {
            if constexpr (FP8) tc_mma_f8(acc, a, b, idesc, more);
            else tc_mma_f16(acc, a, b, idesc, more);
        }
    }
}

__device__ __forceinline__ uint64_t operand_desc(int mn) {
    return mn ? smem_desc_sw128_template(kAtom, 1024) : smem_desc_sw128_template(16, 1024);
}
// Address step of one MMA's K (32 bytes of a K-contiguous row; 16 rows of 128
// bytes of an operand stored along its rows).
__device__ __forceinline__ uint32_t operand_step(int mn) { return mn ? 2048u : 32u; }

// ---------------------------------------------------------------- epilogues
__device__ __forceinline__ void act8(int act, float (&x)[8]) {
    with_act(act, [&](auto a) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = act_fwd<decltype(a)::value>(x[i]);
    });
}

// Up to 8 consecutive columns n.. of output row m, a row to a lane.
template <typename T>
__device__ __forceinline__ void epilogue_row8(const Epilogue& e, bool vec, int64_t m, int64_t n,
                                              int64_t N, float sa, float (&x)[8]) {
    if (n >= N) return;
    const int cnt = int(N - n < 8 ? N - n : 8);
    vec = vec && cnt == 8;
    float t[8];
    if (e.sw) {
        load8<float>(e.sw, n, vec, cnt, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= sa * t[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= sa;
    }
    if (e.bias) {
        load8<T>(e.bias, n, vec, cnt, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] += t[i];
    }
    if (e.Z) store8<T>(e.Z, m * e.ldz + n, vec, cnt, x);
    act8(e.act, x);
    if (e.R) {
        load8<T>(e.R, m * e.ldr + n, vec, cnt, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] += t[i];
    }
    store8<T>(e.Y, m * e.ldy + n, vec, cnt, x);
}

// Up to 8 consecutive rows m.. of output column n, a column to a lane.
template <typename T>
__device__ __forceinline__ void epilogue_col8(const Epilogue& e, int64_t m, int64_t M, int64_t n,
                                              float sw, float bias, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (e.sa && m + i < M) x[i] *= e.sa[m + i];
        x[i] = x[i] * sw + bias;
        if (e.Z && m + i < M) static_cast<T*>(e.Z)[(m + i) * e.ldz + n] = from_f32<T>(x[i]);
    }
    act8(e.act, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (m + i >= M) continue;
        if (e.R) x[i] += to_f32(static_cast<const T*>(e.R)[(m + i) * e.ldr + n]);
        static_cast<T*>(e.Y)[(m + i) * e.ldy + n] = from_f32<T>(x[i]);
    }
}

// ------------------------------------------------------------- tile kernel
// 12 warps: 0 and 2 issue the TMA fills (every other one each), 1 the MMAs (of
// the pair's even CTA) and owns tensor memory, 4..11 run the epilogue, two
// warps to a lane quadrant taking alternate 32-column chunks.
constexpr int kTileThreads = 384;
constexpr int kTileEpiWarps = 8;

struct TileSmem {
    uint8_t* stages;
    uint64_t *full, *empty, *acc_full, *acc_empty, *drain;
    uint32_t* tmem_base;
    volatile int* abort;
};

__device__ __forceinline__ TileSmem carve_tile(uint8_t* raw, const TcLinear& p) {
    TileSmem s;
    uint8_t* b = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    s.stages = b;
    uint64_t* bars = reinterpret_cast<uint64_t*>(b + size_t(p.stages) * (p.p_bytes + p.q_bytes));
    s.full = bars;
    s.empty = bars + p.stages;
    s.acc_full = bars + 2 * p.stages;
    s.acc_empty = s.acc_full + 2;
    s.drain = s.acc_empty + 2;
    s.tmem_base = reinterpret_cast<uint32_t*>(s.drain + 1);
    s.abort = reinterpret_cast<volatile int*>(s.tmem_base + 1);
    return s;
}

// Tile T of the grid: runs of `group` P tiles sweep all Q tiles, odd runs
// backwards, so that the clusters at work share few operand panels in L2.
__device__ __forceinline__ void tile_at(int T, const TcLinear& p, int& tp, int& tq) {
    const int per = p.group * p.tiles_q;
    const int g = T / per;
    const int first = g * p.group;
    const int n = min(p.tiles_p - first, p.group);
    const int r = T - g * per;
    tp = first + r % n;
    tq = r / n;
    if (g & 1) tq = p.tiles_q - 1 - tq;
}

template <typename T, bool SWAP>
__global__ void __launch_bounds__(kTileThreads, 1)
    linear_tile_kernel(const __grid_constant__ CUtensorMap mapP, const __grid_constant__ CUtensorMap mapQ,
                       const __grid_constant__ TcLinear p) {
    extern __shared__ uint8_t smem_raw[];
    const TileSmem s = carve_tile(smem_raw, p);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = int(cluster_ctarank());
    const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;
    const uint32_t stage_bytes = p.p_bytes + p.q_bytes;
    const uint64_t tmo = p.timeout_ns;
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&mapP);
        prefetch_tensormap(&mapQ);
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.acc_full[i], 1);
            mbar_init(&s.acc_empty[i], 2 * kTileEpiWarps);  // both CTAs' epilogue warps
        }
        mbar_init(s.drain, 1);
        *s.abort = 0;
        fence_mbarrier_init();
    }
    if (warp == 1) {
        tmem_alloc<2>(s.tmem_base, 512);
        tmem_relinquish_alloc_permit<2>();
    }
    tc_fence_before_sync();
    cluster_sync();  // no fill or arrival reaches a peer's barrier before it exists
    tc_fence_after_sync();
    grid_launch_dependents();
    const uint32_t tmem = *s.tmem_base;
    uint32_t issued_any = 0, issued_parity = 0;  // a producer's last fill of each stage

    const int prod = warp == 0 ? 0 : (warp == 2 ? 1 : -1);
    if (prod >= 0 && lane == 0) {
        grid_dependency_wait();
        const uint64_t pol = l2_policy(2);  // panels are read again by later tiles
        const int q_rows = p.bn / 2;
        const int q_atoms = (q_rows + 63) / 64;
        const uint32_t tx = 2u * (p.p_bytes + (p.q_mn ? uint32_t(q_atoms) * kAtom : uint32_t(q_rows) * 128u));
        int stage = 0, turn = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = cid; ok && t < p.tiles; t += ncl) {
            int tp, tq;
            tile_at(t, p, tp, tq);
            const int p0 = (2 * tp + rank) * 128;
            const int q0 = tq * p.bn + rank * q_rows;
            for (int kb = 0; kb < p.k_blocks; ++kb, turn ^= 1) {
                if (turn == prod) {
                    if (!wait_bounded(&s.empty[stage], phase ^ 1u, s.abort, tmo)) {
                        ok = false;
                        break;
                    }
                    uint8_t* sp = s.stages + size_t(stage) * stage_bytes;
                    uint8_t* sq = sp + p.p_bytes;
                    const int k0 = kb * p.bk;
                    const uint32_t fb = mapa_shared(smem_u32(&s.full[stage]), 0);
                    if (rank == 0) mbar_arrive_expect_tx(&s.full[stage], tx);
                    if (p.p_mn) {
                        tma_load_2d_pair_hint(sp, &mapP, fb, p0, k0, pol);
                        tma_load_2d_pair_hint(sp + kAtom, &mapP, fb, p0 + 64, k0, pol);
                    } else {
                        tma_load_2d_pair_hint(sp, &mapP, fb, k0, p0, pol);
                    }
                    if (p.q_mn) {
                        for (int a = 0; a < q_atoms; ++a)
                            tma_load_2d_pair_hint(sq + a * kAtom, &mapQ, fb, q0 + 64 * a, k0, pol);
                    } else {
                        tma_load_2d_pair_hint(sq, &mapQ, fb, k0, q0, pol);
                    }
                    issued_any |= 1u << stage;
                    issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
                }
                if (++stage == p.stages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
    }
    if (warp == 1 && lane == 0 && rank == 0) {
        const uint64_t dP = operand_desc(p.p_mn), dQ = operand_desc(p.q_mn);
        const uint32_t step_p = operand_step(p.p_mn), step_q = operand_step(p.q_mn);
        const uint32_t base = smem_u32(s.stages), p_bytes = p.p_bytes, idesc = p.idesc;
        const int nstages = p.stages, nk = p.k_blocks;
        const bool fp8 = p.fp8 != 0;
        int stage = 0, it = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = cid; ok && t < p.tiles; t += ncl, ++it) {
            const int b = it & 1;
            if (!wait_bounded(&s.acc_empty[b], ((it >> 1) & 1) ^ 1u, s.abort, tmo)) break;
            tc_fence_after_sync();
            const uint32_t acc = tmem + uint32_t(b) * 256u;
            for (int kb = 0; kb < nk; ++kb) {
                if (!wait_bounded(&s.full[stage], phase, s.abort, tmo)) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t ap = base + uint32_t(stage) * stage_bytes;
                if (fp8)
                    issue_stage<true, true>(acc, dP, dQ, ap, ap + p_bytes, step_p, step_q, idesc, kb == 0);
                else
                    issue_stage<true, false>(acc, dP, dQ, ap, ap + p_bytes, step_p, step_q, idesc, kb == 0);
                tc_commit_pair_multicast(&s.empty[stage], 3);
                if (++stage == nstages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (ok) tc_commit_pair_multicast(&s.acc_full[b], 3);
        }
        tc_commit_pair(s.drain);
        wait_bounded(s.drain, 0, s.abort, tmo, true);
    }
    if (warp >= 4) {
        grid_dependency_wait();
        const int quad = warp & 3, half = (warp - 4) >> 2;
        const uint32_t lanes = uint32_t(quad * 32) << 16;
        const int chunks = p.bn / 32;
        int it = 0;
        for (int t = cid; t < p.tiles; t += ncl, ++it) {
            int tp, tq;
            tile_at(t, p, tp, tq);
            const int64_t pr = int64_t(2 * tp + rank) * 128 + quad * 32 + lane;
            const int64_t q0 = int64_t(tq) * p.bn;
            const int b = it & 1;
            bool ok = wait_bounded(&s.acc_full[b], (it >> 1) & 1, s.abort, tmo);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after_sync();
            const bool live = pr < p.Mp;
            // Swapped: this lane's output column; normal: its output row.
            const float sa = !SWAP && live && p.e.sa ? p.e.sa[pr] : 1.f;
            const float sw = SWAP && live && p.e.sw ? p.e.sw[pr] : 1.f;
            const float bias = SWAP && live && p.e.bias ? to_f32(static_cast<const T*>(p.e.bias)[pr]) : 0.f;
            const int limit = int(min(int64_t(p.bn), p.Nq - q0));  // columns in the matrix
            const uint32_t acc = tmem + lanes + uint32_t(b * 256);
            // 32-column chunks half, half + 2, ...
            for (int c = 32 * half; c < limit; c += 64) {
                uint32_t r[32];
                tmem_ld_32x32b_x32(acc + uint32_t(c), r);
                tmem_ld_wait(r);
                if (live) {
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        float x[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(r[8 * g + i]);
                        if constexpr (SWAP)
                            epilogue_col8<T>(p.e, q0 + c + 8 * g, p.Nq, pr, sw, bias, x);
                        else
                            epilogue_row8<T>(p.e, p.vec, pr, q0 + c + 8 * g, p.Nq, sa, x);
                    }
                }
                __syncwarp();
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&s.acc_empty[b]), 0));
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    if (*s.abort) {
        // Both CTAs' fills complete on the even CTA's barriers.
        if (prod >= 0 && lane == 0 && rank == 0)
            for (int i = 0; i < p.stages; ++i)
                if (issued_any & (1u << i))
                    wait_bounded(&s.full[i], (issued_parity >> i) & 1u, s.abort, tmo, true);
        __syncthreads();
    }
    cluster_sync();  // no CTA leaves while its peer may still reach its barriers
    if (warp == 1) {
        __syncwarp();
        tc_fence_after_sync();
        tmem_dealloc<2>(tmem, 512);
    }
}

// ------------------------------------------------------------ split kernel
constexpr int kSplitThreads = 256;
constexpr int kPad = 129;  // words between a column's and the next one's 128 lanes

struct SplitSmem {
    uint8_t* stages;  // then the partial sums, [bn][kPad] f32
    uint64_t *full, *empty, *acc_full;
    uint32_t* tmem_base;
    volatile int* abort;
};

__device__ __forceinline__ SplitSmem carve_split(uint8_t* raw, const TcLinear& p) {
    SplitSmem s;
    uint8_t* b = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    s.stages = b;
    uint64_t* bars = reinterpret_cast<uint64_t*>(b + p.ring_bytes);
    s.full = bars;
    s.empty = bars + p.stages;
    s.acc_full = bars + 2 * p.stages;
    s.tmem_base = reinterpret_cast<uint32_t*>(s.acc_full + 1);
    s.abort = reinterpret_cast<volatile int*>(s.tmem_base + 1);
    return s;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

template <typename T, bool SWAP>
__global__ void __launch_bounds__(kSplitThreads, 1)
    linear_split_kernel(const __grid_constant__ CUtensorMap mapP, const __grid_constant__ CUtensorMap mapQ,
                        const __grid_constant__ TcLinear p) {
    extern __shared__ uint8_t smem_raw[];
    const SplitSmem s = carve_split(smem_raw, p);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = int(cluster_ctarank());
    const int tile = blockIdx.x / p.split;
    const int tp = tile % p.tiles_p, tq = tile / p.tiles_p;
    const int p0 = tp * p.bp, q0 = tq * p.bn;
    const int kb0 = int(int64_t(p.k_blocks) * rank / p.split);
    const int kb1 = int(int64_t(p.k_blocks) * (rank + 1) / p.split);
    const uint32_t stage_bytes = p.p_bytes + p.q_bytes;
    const uint64_t tmo = p.timeout_ns;
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&mapP);
        prefetch_tensormap(&mapQ);
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        mbar_init(s.acc_full, 1);
        *s.abort = 0;
        fence_mbarrier_init();
    }
    if (warp == 1) {
        tmem_alloc<1>(s.tmem_base, uint32_t(p.tmem_cols));
        tmem_relinquish_alloc_permit<1>();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    grid_launch_dependents();
    const uint32_t tmem = *s.tmem_base;
    uint32_t issued_any = 0, issued_parity = 0;
    if (warp == 0 && lane == 0) {
        grid_dependency_wait();
        const uint64_t pol_p = l2_policy(p.tiles_q == 1 ? 1 : 2), pol_q = l2_policy(2);
        const int q_atoms = (p.bn + 63) / 64, p_atoms = (p.bp + 63) / 64;
        const uint32_t tx = (p.p_mn ? uint32_t(p_atoms) * kAtom : uint32_t(p.bp) * 128u) +
                            (p.q_mn ? uint32_t(q_atoms) * kAtom : uint32_t(p.bn) * 128u);
        int stage = 0;
        uint32_t phase = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!wait_bounded(&s.empty[stage], phase ^ 1u, s.abort, tmo)) break;
            uint8_t* sp = s.stages + size_t(stage) * stage_bytes;
            uint8_t* sq = sp + p.p_bytes;
            const int k0 = kb * p.bk;
            mbar_arrive_expect_tx(&s.full[stage], tx);
            if (p.p_mn) {
                for (int a = 0; a < p_atoms; ++a)
                    tma_load_2d_hint(sp + a * kAtom, &mapP, &s.full[stage], p0 + 64 * a, k0, pol_p);
            } else {
                tma_load_2d_hint(sp, &mapP, &s.full[stage], k0, p0, pol_p);
            }
            if (p.q_mn) {
                for (int a = 0; a < q_atoms; ++a)
                    tma_load_2d_hint(sq + a * kAtom, &mapQ, &s.full[stage], q0 + 64 * a, k0, pol_q);
            } else {
                tma_load_2d_hint(sq, &mapQ, &s.full[stage], k0, q0, pol_q);
            }
            issued_any |= 1u << stage;
            issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
            if (++stage == p.stages) {
                stage = 0;
                phase ^= 1u;
            }
        }
    } else if (warp == 1 && lane == 0) {
        const uint64_t dP = operand_desc(p.p_mn), dQ = operand_desc(p.q_mn);
        const uint32_t step_p = operand_step(p.p_mn), step_q = operand_step(p.q_mn);
        const uint32_t base = smem_u32(s.stages), p_bytes = p.p_bytes, idesc = p.idesc;
        const int nstages = p.stages;
        const bool fp8 = p.fp8 != 0;
        int stage = 0;
        uint32_t phase = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!wait_bounded(&s.full[stage], phase, s.abort, tmo)) break;
            tc_fence_after_sync();
            const uint32_t ap = base + uint32_t(stage) * stage_bytes;
            if (fp8)
                issue_stage<false, true>(tmem, dP, dQ, ap, ap + p_bytes, step_p, step_q, idesc, kb == kb0);
            else
                issue_stage<false, false>(tmem, dP, dQ, ap, ap + p_bytes, step_p, step_q, idesc, kb == kb0);
            tc_commit(&s.empty[stage]);
            if (++stage == nstages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        // Complete once every MMA issued is (also after a wait gave up).
        tc_commit(s.acc_full);
    }
    __syncwarp();
    // Every warp waits for the MMAs before it may read tensor memory, reuse the
    // stages or leave.
    bool ok = wait_bounded(s.acc_full, 0, s.abort, tmo, true);
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after_sync();
    float* part = reinterpret_cast<float*>(s.stages);
    if (ok && !*s.abort) {
        const int quad = warp & 3;
        for (int c = warp >> 2; 32 * c < p.bn; c += 2) {
            uint32_t r[32];
            tmem_ld_32x32b_x32(tmem + (uint32_t(quad * 32) << 16) + uint32_t(32 * c), r);
            tmem_ld_wait(r);
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (32 * c + i < p.bn)
                    part[(32 * c + i) * kPad + quad * 32 + lane] = __uint_as_float(r[i]);
        }
    }
    tc_fence_before_sync();
    __syncwarp();
    cluster_sync();
    grid_dependency_wait();
    if (!*s.abort) {
        // This CTA's share of the tile: every split-th run of 32 outputs along
        // the output's rows' contiguous direction. Ranks are added in order.
        const uint32_t mine = smem_u32(part);
        const int runs_in = SWAP ? (p.bp + 31) / 32 : (p.bn + 31) / 32;  // runs along that direction
        const int lines = SWAP ? p.bn : p.bp;
        with_act(p.e.act, [&](auto act) {
            constexpr int ACT = decltype(act)::value;
            for (int i = warp * p.split + rank; i < runs_in * lines; i += p.split * (kSplitThreads / 32)) {
                const int along = 32 * (i % runs_in) + lane, line = i / runs_in;
                const int pl = SWAP ? along : line, ql = SWAP ? line : along;
                if (pl >= p.bp || ql >= p.bn || p0 + pl >= p.Mp || q0 + ql >= p.Nq) continue;
                const uint32_t at = mine + 4u * uint32_t(ql * kPad + pl);
                float x = 0.f;
                for (int r = 0; r < p.split; ++r) x += ld_cluster_f32(mapa_shared(at, uint32_t(r)));
                if constexpr (SWAP)
                    epilogue_one<T, ACT>(p.e, q0 + ql, p0 + pl, x);
                else
                    epilogue_one<T, ACT>(p.e, p0 + pl, q0 + ql, x);
            }
        });
    }
    if (*s.abort && warp == 0 && lane == 0)
        for (int i = 0; i < p.stages; ++i)
            if (issued_any & (1u << i))
                wait_bounded(&s.full[i], (issued_parity >> i) & 1u, s.abort, tmo, true);
    __syncwarp();
    cluster_sync();  // peers have read this CTA's partial sums
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc<1>(tmem, uint32_t(p.tmem_cols));
    }
}

using TcFn = void (*)(CUtensorMap, CUtensorMap, TcLinear);

template <typename T>
TcFn pick_typed(const TcLinear& p) {
    if (p.pair) return p.swap ? linear_tile_kernel<T, true> : linear_tile_kernel<T, false>;
    return p.swap ? linear_split_kernel<T, true> : linear_split_kernel<T, false>;
}

TcFn pick(const TcLinear& p) {
    if (p.e.out == TPGEMM_ELEM_F16) return pick_typed<__half>(p);
    if (p.e.out == TPGEMM_ELEM_BF16) return pick_typed<__nv_bfloat16>(p);
    return pick_typed<float>(p);
}

}  // namespace

size_t tc_linear_smem(const TcLinear& p) {
    const size_t ring = p.pair ? size_t(p.stages) * (p.p_bytes + p.q_bytes) : size_t(p.ring_bytes);
    return 1024 + ring + 8 * (2 * size_t(p.stages) + 5) + 16;
}

cudaError_t launch_tc_linear(const CUtensorMap& mapP, const CUtensorMap& mapQ, const TcLinear& p,
                             int grid, cudaStream_t stream) {
    const int cluster = p.pair ? 2 : p.split;
    if (p.stages < 2 || p.stages > 32 || grid % cluster != 0 || p.bn % 16 != 0 || p.bn > 256 ||
        (p.pair && (p.bn % 32 != 0 || p.group < 1)) ||
        (!p.pair && (p.bp > 128 || p.bp % 16 != 0 || p.split < 1 || p.split > 8 ||
                     p.split > p.k_blocks ||
                     size_t(p.bn) * kPad * 4 > p.ring_bytes ||
                     size_t(p.stages) * (p.p_bytes + p.q_bytes) > p.ring_bytes)))
        return cudaErrorInvalidValue;
    const size_t smem = tc_linear_smem(p);
    if (smem > size_t(kTcMaxSmem)) return cudaErrorInvalidConfiguration;
    const TcFn fn = pick(p);
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcMaxSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(p.pair ? kTileThreads : kSplitThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(cluster);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fn, mapP, mapQ, p);
}

cudaError_t tc_linear_max_pairs(const TcLinear& p, int* pairs) {
    const TcFn fn = pick(p);
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcMaxSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = tc_linear_smem(p);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaOccupancyMaxActiveClusters(pairs, fn, &cfg);
}

cudaError_t linear_read_and_clear_status(int* status) {
    cudaError_t e = cudaMemcpyFromSymbol(status, g_linear_status, sizeof(int));
    const int zero = 0;
    if (e == cudaSuccess && *status) e = cudaMemcpyToSymbol(g_linear_status, &zero, sizeof(int));
    return e;
}

}  // namespace tpg
