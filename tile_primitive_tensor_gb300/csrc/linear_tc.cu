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
// The gated layer's products take half of a tile's weight rows from W's first
// half and half from its second, so that an output's gate and factor meet in one
// tile: in a pair each CTA loads one half's rows as its share of Q, and elsewhere
// the weights' box comes as two.
//
// Operands are read where they lie, K-contiguous or along their rows, by TMA
// into 128-byte-swizzled stages (K's and the rows' ends read as zero). The tensor
// cores add into their 32-bit accumulators with truncation: against 64 bits a
// sum of random signs is off by 5e-7 of its size at K = 512, 2e-6 at 4096 and
// 9e-6 at 16384 (shares of a split K are added with rounding and are each that
// much shorter). 16-bit outputs do not see it; taking the sums out of tensor
// memory every 1024 of K, for 32-bit ones, would halve the tile's width. Every
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

constexpr uint32_t kAtom = 8192;  // an operand stored along its rows: 64 K x 64 rows of 16 bits

// Waits for a phase of `bar` for at most timeout_ns from when the previous grid has
// ended: abort[1] is set once a thread of this CTA has passed the dependency. (The
// check costs a wait nothing until it expires. With the dependency in every warp
// before its first wait, a norm and its product took 15.0 us for 14.7: the MMA
// warp's instructions came that much later.)
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, volatile int* abort,
                                             uint64_t timeout_ns, bool drain = false) {
    if (mbar_try_wait(bar, parity)) return true;
    uint64_t t0 = globaltimer_ns();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (!drain && *abort) return false;
        if (globaltimer_ns() - t0 > timeout_ns) {
            if (!abort[1]) {
                t0 = globaltimer_ns();
                continue;
            }
            *abort = 1;
            atomicExch(&g_linear_status, kStatusTimeout);
            return false;
        }
    }
}

// Four MMAs, one 128-byte-wide stage of K, and their commit to `bar`, issued by
// one thread that the warp elects. The whole warp runs this, convergent, with
// the same values: descriptors, addresses and flags then live in uniform
// registers, where the MMA takes them from. (Under a one-lane branch each MMA's
// operands are moved there one by one, which cost about 135 cycles an MMA, more
// than the 128 it computes for at 256 x 256: 4096^3 bf16 88 us against 74.)
// a, b: descriptors of the stage's operands; step_a, step_b: their step for one
// MMA's K. mask: the CTAs whose barrier the commit reaches (pair form).
#define TPG_STAGE_ASM(KIND, CG, COMMIT)                                                   \
    asm volatile(                                                                         \
        "{\n\t.reg .pred e, p, t;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"                \
        "elect.sync _|e, 0xffffffff;\n\t"                                                 \
        "setp.ne.b32 p, %6, 0;\n\t"                                                       \
        "setp.eq.b32 t, 0, 0;\n\t"                                                        \
        "add.u64 a1, %1, %3;\n\tadd.u64 b1, %2, %4;\n\t"                                  \
        "add.u64 a2, a1, %3;\n\tadd.u64 b2, b1, %4;\n\t"                                  \
        "add.u64 a3, a2, %3;\n\tadd.u64 b3, b2, %4;\n\t"                                  \
        "@e tcgen05.mma.cta_group::" CG ".kind::" KIND " [%0], %1, %2, %5, p;\n\t"        \
        "@e tcgen05.mma.cta_group::" CG ".kind::" KIND " [%0], a1, b1, %5, t;\n\t"        \
        "@e tcgen05.mma.cta_group::" CG ".kind::" KIND " [%0], a2, b2, %5, t;\n\t"        \
        "@e tcgen05.mma.cta_group::" CG ".kind::" KIND " [%0], a3, b3, %5, t;\n\t"        \
        "@e " COMMIT "\n\t}" ::"r"(acc),                                                  \
        "l"(a), "l"(b), "l"(step_a), "l"(step_b), "r"(idesc), "r"(more), "r"(bar), "h"(mask) \
        : "memory")

template <bool PAIR>
__device__ __forceinline__ void issue_stage(bool fp8, uint32_t acc, uint64_t a, uint64_t b,
                                            uint64_t step_a, uint64_t step_b, uint32_t idesc,
                                            uint32_t more, uint32_t bar, uint16_t mask) {
    if constexpr (PAIR) {
        if (fp8)
            TPG_STAGE_ASM("f8f6f4", "2",
                          "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
                          ".multicast::cluster.b64 [%7], %8;");
        else
            TPG_STAGE_ASM("f16", "2",
                          "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
                          ".multicast::cluster.b64 [%7], %8;");
    } else {
        if (fp8)
            TPG_STAGE_ASM("f8f6f4", "1",
                          "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%7];");
        else
            TPG_STAGE_ASM("f16", "1",
                          "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%7];");
    }
}
#undef TPG_STAGE_ASM

// TMA loads and their byte counts, issued likewise by the elected thread of a
// convergent warp: a fill of two boxes from under a one-lane branch held its
// thread for 400 clocks, most of the 512 that a 256 x 256 stage computes for.
__device__ __forceinline__ void expect_elected(uint32_t bar, uint32_t bytes) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
        "r"(bytes)
        : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void load_elected(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x,
                                             int32_t y, uint64_t policy) {
    if constexpr (PAIR)
        asm volatile(
            "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
            "@e cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
            ".L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;\n\t}" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "l"(policy)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
            "@e cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
            ".L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;\n\t}" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "l"(policy)
            : "memory");
}

__device__ __forceinline__ void prefetch_elected(const CUtensorMap* map, int32_t x, int32_t y) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];\n\t}" ::"l"(
            reinterpret_cast<uint64_t>(map)),
        "r"(x), "r"(y)
        : "memory");
}

// One operand's box or boxes of a stage: `rows` rows from r0 on, K from k0 on.
template <bool PAIR>
__device__ __forceinline__ void load_operand(uint32_t dst, const CUtensorMap* map, uint32_t bar, int mn,
                                             int atoms, int r0, int k0, uint64_t policy) {
    if (mn) {
        for (int a = 0; a < atoms; ++a)
            load_elected<PAIR>(dst + uint32_t(a) * kAtom, map, bar, r0 + 64 * a, k0, policy);
    } else {
        load_elected<PAIR>(dst, map, bar, k0, r0, policy);
    }
}

__device__ __forceinline__ void st_cluster_b32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Commits of the elected thread's MMAs (the whole warp, convergent).
__device__ __forceinline__ void commit_elected(uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void commit_elected_pair(uint64_t* bar, uint16_t mask) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
        "h"(mask)
        : "memory");
}

__device__ __forceinline__ uint64_t operand_desc(int mn) {
    return mn ? smem_desc_sw128_template(kAtom, 1024) : smem_desc_sw128_template(16, 1024);
}
// Descriptor step (16-byte units) of one MMA's K: 32 bytes of a K-contiguous
// row; 16 rows of 128 bytes of an operand stored along its rows.
__device__ __forceinline__ uint64_t operand_step(int mn) { return mn ? 128u : 2u; }

// ---------------------------------------------------------------- epilogues
// The activation of N values on their way to outputs of type T.
template <typename T, int N>
__device__ __forceinline__ void act_n(int act, float (&x)[N]) {
    with_act(act, [&](auto a) {
#pragma unroll
        for (int i = 0; i < N; i += 2)
            split(act_fwd<decltype(a)::value, sizeof(T) == 4>(f2(x[i], x[i + 1])), x[i], x[i + 1]);
    });
}

// x[i] of lane j and x[j] of lane i change places.
template <typename V>
__device__ __forceinline__ void transpose32(int lane, V (&x)[32]) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
        const bool high = (lane & s) != 0;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            if (i & s) continue;
            const V got = __shfl_xor_sync(0xffffffffu, high ? x[i] : x[i + s], s);
            if (high) x[i] = got;
            else x[i + s] = got;
        }
    }
}

// A 32 x 32 chunk, a row m0 + lane to a lane with that row's scale sa, of
// outputs whose rows start anywhere: turned, so that a warp reads and writes 32
// neighbouring columns of a row at a time.
template <typename T>
__device__ __forceinline__ void epilogue_turned(const Epilogue& e, int64_t m0, int64_t n0, int64_t M, int64_t N,
                                                int lane, float sa, float (&x)[32]) {
    const int64_t n = n0 + lane;
    const int rows = int(min(int64_t(32), M - m0));
    T res[32];  // asked for before anything that it is not needed for
    if (e.R && n < N) {
        const T* r = static_cast<const T*>(e.R) + m0 * e.ldr + n;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < rows) res[i] = r[i * e.ldr];
    }
    transpose32(lane, x);
    if (e.sa) {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] *= __shfl_sync(0xffffffffu, sa, i);
    }
    if (n < N) {
        const float sw = e.sw ? e.sw[n] : 1.f;
        const float bias = e.bias ? to_f32(static_cast<const T*>(e.bias)[n]) : 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = fmaf(x[i], sw, bias);
        if (e.Z) {
            T* z = static_cast<T*>(e.Z) + m0 * e.ldz + n;
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i < rows) z[i * e.ldz] = from_f32<T>(x[i]);
        }
        act_n<T>(e.act, x);
        if (e.R) {
            float r[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = i < rows ? to_f32(res[i]) : 0.f;
            add_residual<T>(e.rest, r, x);
        }
        T* y = static_cast<T*>(e.Y) + m0 * e.ldy + n;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < rows) y[i * e.ldy] = from_f32<T>(x[i]);
    }
    __syncwarp();
}

// The same of the gated layer: x the gates' sums, u the factors'.
template <typename T>
__device__ __forceinline__ void epilogue_turned_gated(const Epilogue& e, int64_t m0, int64_t n0, int64_t M,
                                                      int64_t N, int lane, float sa, float (&x)[32],
                                                      float (&u)[32]) {
    const int64_t n = n0 + lane;
    const int rows = int(min(int64_t(32), M - m0));
    transpose32(lane, x);
    transpose32(lane, u);
    if (e.sa) {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float f = __shfl_sync(0xffffffffu, sa, i);
            x[i] *= f;
            u[i] *= f;
        }
    }
    if (n < N) {
        const float swx = e.sw ? e.sw[n] : 1.f, swu = e.sw ? e.sw[N + n] : 1.f;
        const float bx = e.bias ? to_f32(static_cast<const T*>(e.bias)[n]) : 0.f;
        const float bu = e.bias ? to_f32(static_cast<const T*>(e.bias)[N + n]) : 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            x[i] = fmaf(x[i], swx, bx);
            u[i] = fmaf(u[i], swu, bu);
        }
        if (e.Z) {
            T* z = static_cast<T*>(e.Z) + m0 * e.ldz + n;
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i < rows) {
                    z[i * e.ldz] = from_f32<T>(x[i]);
                    z[i * e.ldz + N] = from_f32<T>(u[i]);
                }
        }
        act_n<T>(e.act, x);
        T* y = static_cast<T*>(e.Y) + m0 * e.ldy + n;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (i < rows) y[i * e.ldy] = from_f32<T>(x[i] * u[i]);
    }
    __syncwarp();
}

// 32 columns of an output row, staged for a TMA store: a lane's row of the
// warp's 32 x 32 tile, its 16-byte units placed by the store's swizzle (64
// bytes to a row of 16-bit outputs, 128 to one of 32-bit ones).
template <typename T>
__device__ __forceinline__ uint4* staged_unit(uint8_t* buf, int lane, int u) {
    if constexpr (sizeof(T) == 4)
        return reinterpret_cast<uint4*>(buf + lane * 128) + (u ^ (lane & 7));
    else
        return reinterpret_cast<uint4*>(buf + lane * 64) + (u ^ ((lane >> 1) & 3));
}

template <typename T>
__device__ __forceinline__ void stage_row32(uint8_t* buf, int lane, const float (&x)[32]) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = x[8 * g + i];
        if constexpr (sizeof(T) == 4) {
            *staged_unit<T>(buf, lane, 2 * g) = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]),
                                                           __float_as_uint(f[2]), __float_as_uint(f[3]));
            *staged_unit<T>(buf, lane, 2 * g + 1) = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]),
                                                               __float_as_uint(f[6]), __float_as_uint(f[7]));
        } else {
            *staged_unit<T>(buf, lane, g) = pack8<T>(f);
        }
    }
}

template <typename T>
__device__ __forceinline__ void add_staged32(uint8_t* buf, int lane, int rest, float (&x)[32]) {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        float f[8];
        if constexpr (sizeof(T) == 4) {
            const uint4 a = *staged_unit<T>(buf, lane, 2 * g), b = *staged_unit<T>(buf, lane, 2 * g + 1);
            f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y);
            f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
            f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y);
            f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
        } else {
            unpack8<T>(*staged_unit<T>(buf, lane, g), f);
        }
        add_residual<T>(rest, f, x + 8 * g);
    }
}

// x += / *= the 32 values that the lanes hold, one to a column.
template <bool MUL>
__device__ __forceinline__ void apply_columns(float v, float (&x)[32]) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
        const F2 a = f2(x[i], x[i + 1]);
        const F2 c = f2(__shfl_sync(0xffffffffu, v, i), __shfl_sync(0xffffffffu, v, i + 1));
        split(MUL ? mul(a, c) : add(a, c), x[i], x[i + 1]);
    }
}

// ------------------------------------------------------------- tile kernel
// 12 warps: 0 and 2 issue the TMA fills (every other one each), 1 the MMAs (of
// a pair's even CTA) and owns tensor memory, 4..11 run the epilogue, two warps
// to a lane quadrant taking alternate 32-column chunks.
//
// A stage brings 128 P rows and bn / 2 Q rows of 128 bytes into each SM, which
// takes in 64 bytes a clock: 256 + bn clocks, against 2 bn at the tensor rate.
// So bn = 256 is where both meet (515 measured), and narrower tiles are bound
// by delivery (413 at 128). Two pairs sharing a tile by TMA multicast measured
// no faster: they save reads of L2, not what arrives at an SM.
//
// Outputs whose rows start on 16-byte boundaries leave through a staging tile
// and TMA stores; the residual comes in the same way, ahead of its use. Stores
// straight from registers, 16 bytes to each of 32 rows, occupy the load/store
// path for 32 cycles an instruction, and those of single elements as long: the
// other outputs are turned first (2048 x 4099 x 2048 bf16: 86 -> 28 us). With Z and a
// residual the buffers hold Z and Y, and the residual is read that way, 16 bytes to
// each of 32 rows (4096^3 bf16 with gelu: plain 78.2 us, Z 80.1, residual 80.4, both
// 84.2).
constexpr int kTileThreads = 384;
constexpr int kTileEpiWarps = 8;
constexpr int kStaging = 4096;  // staging bytes of an epilogue warp
constexpr int kBiasBytes = 256;

struct TileSmem {
    uint8_t* stages;
    uint8_t* staging;
    uint8_t* bias;  // [epilogue warps][128] 16-bit bias of the warp's columns
    uint64_t *full, *empty, *acc_full, *acc_empty, *drain, *rbar;
    uint32_t* tmem_base;
    volatile int* abort;  // and [1], see wait_bounded
    volatile int* fills;  // after a timeout: the two producers' fills,
    volatile int* peer;   // and the other CTA's, [2] set once it has given up too
};

__device__ __forceinline__ TileSmem carve_tile(uint8_t* raw, const TcLinear& p) {
    TileSmem s;
    uint8_t* b = raw;  // 1024-byte aligned
    s.stages = b;
    s.staging = b + size_t(p.stages) * (p.p_bytes + p.q_bytes);
    s.bias = s.staging + kTileEpiWarps * kStaging;
    uint64_t* bars = reinterpret_cast<uint64_t*>(s.bias + kTileEpiWarps * kBiasBytes);
    s.full = bars;
    s.empty = bars + p.stages;
    s.acc_full = bars + 2 * p.stages;
    s.acc_empty = s.acc_full + 2;
    s.drain = s.acc_empty + 2;
    s.rbar = s.drain + 1;  // [epilogue warps][2] residual fills
    s.tmem_base = reinterpret_cast<uint32_t*>(s.rbar + 2 * kTileEpiWarps);
    s.abort = reinterpret_cast<volatile int*>(s.tmem_base + 1);
    s.fills = s.abort + 2;
    s.peer = s.fills + 2;
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

// Lets the fills of a pair that gave up land, by a thread of the even CTA, on
// whose barriers they complete. Fill g (of stage g % stages, by producer g & 1) is
// both CTAs' boxes, but one CTA may have stopped a fill before the other: the
// half that does not come is left out of the count.
__device__ __forceinline__ void drain_fills(const TileSmem& s, const TcLinear& p, uint32_t half, uint64_t tmo) {
    const int own0 = s.fills[0], own1 = s.fills[1], peer0 = s.peer[0], peer1 = s.peer[1];
    const int end = max(2 * max(own0, peer0) - 1, 2 * max(own1, peer1));  // past the last fill
    // A stage's last fill is among the last 2 stages + 2: producers stay within
    // the ring of each other.
    uint32_t seen = 0;
    for (int g = end - 1; g >= 0 && g >= end - 2 * p.stages - 2; --g) {
        const int i = g % p.stages;
        const bool ours = (g >> 1) < ((g & 1) ? own1 : own0), theirs = (g >> 1) < ((g & 1) ? peer1 : peer0);
        if (((seen >> i) & 1u) || !(ours || theirs)) continue;
        seen |= 1u << i;
        if (!ours) mbar_arrive_expect_tx(&s.full[i], half);
        if (!theirs)
            asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(&s.full[i])),
                         "r"(half)
                         : "memory");
        wait_bounded(&s.full[i], uint32_t(g / p.stages) & 1u, s.abort, tmo, true);
    }
}

// The epilogue warps of a gated product. A tile's columns [0, bn / 2) hold gates
// and the others their factors; a warp takes 32 of both at a time and stores the
// 32 products, and ahead of them, when Z is kept, the two 32 that they come from.
template <typename T>
__device__ __forceinline__ void gated_epilogue(const TcLinear& p, const TileSmem& s, const CUtensorMap& mapY,
                                               const CUtensorMap& mapZ, const CUtensorMap& mapZu, uint32_t tmem,
                                               int warp, int lane, int rank, int cid, int ncl) {
    const Epilogue& e = p.e;
    const int ew = warp - 4, quad = warp & 3, half = ew >> 2, width = p.bn / 2;
    const uint32_t lanes = uint32_t(quad * 32) << 16;
    uint8_t* const staging = s.staging + ew * kStaging;
    constexpr int kBuf = 1024 * int(sizeof(T));  // one 32 x 32 tile
    constexpr int kBufs = kStaging / kBuf;       // 2, or 1 of 32-bit outputs
    const bool tma = p.tma_out != 0;
    const uint64_t pol = l2_policy(1);  // outputs pass through once
    int j = 0;                          // the buffer of the next store
    const auto emit = [&](const CUtensorMap& map, const float (&v)[32], int64_t n, int64_t m) {
        if (lane == 0) bulk_wait_group_read<kBufs - 1>();  // the buffer's last store has been read
        __syncwarp();
        stage_row32<T>(staging + j * kBuf, lane, v);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_2d_hint(&map, staging + j * kBuf, int(n), int(m), pol);
            bulk_commit_group();
        }
        j ^= kBufs - 1;
    };
    for (int t = cid, it = 0; t < p.tiles; t += ncl, ++it) {
        int tp, tq;
        tile_at(t, p, tp, tq);
        const int64_t m0 = int64_t(2 * tp + rank) * 128 + quad * 32, m = m0 + lane;
        const int64_t n0 = int64_t(tq) * width;
        const int b = it & 1;
        // This warp's chunks: columns c = 32 half, + 64, ... below limit.
        const int limit = m0 < p.Mp ? int(max(int64_t(0), min(int64_t(width), p.Nq - n0))) : 0;
        const float sa = m < p.Mp && e.sa ? e.sa[m] : 1.f;
        // As of the plain epilogue: a 16-bit bias in shared memory, a 32-bit one and
        // the columns' scales in registers, a chunk ahead.
        constexpr bool kBiasSmem = sizeof(T) == 2;
        T* const bias_s = reinterpret_cast<T*>(s.bias + ew * kBiasBytes);  // [chunk][half of W][32]
        float bias_c[2] = {0.f, 0.f}, sw_c[2] = {1.f, 1.f};
        const auto fetch_columns = [&](int c) {
            const int64_t n = n0 + c + lane;
            if (c >= limit || n >= p.Nq) return;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!kBiasSmem && e.bias) bias_c[h] = to_f32(static_cast<const T*>(e.bias)[n + h * p.Nq]);
                if (e.sw) sw_c[h] = e.sw[n + h * p.Nq];
            }
        };
        if (tma) {
            if (kBiasSmem && e.bias) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int c = 32 * half + 64 * (i >> 1);
                    const int64_t n = n0 + c + lane;
                    if (c < limit && n < p.Nq)
                        bias_s[32 * i + lane] = static_cast<const T*>(e.bias)[n + (i & 1) * p.Nq];
                }
                __syncwarp();
            }
            fetch_columns(32 * half);
        }
        bool ok = wait_bounded(&s.acc_full[b], (it >> 1) & 1, s.abort, p.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after_sync();
        const uint32_t acc = tmem + lanes + uint32_t(b * 256);
        for (int c = 32 * half; c < limit; c += 64) {
            float x[2][32];  // gates, factors
            {
                uint32_t r[32], q[32];
                tmem_ld_32x32b_x32(acc + uint32_t(c), r);
                tmem_ld_32x32b_x32(acc + uint32_t(width + c), q);
                tmem_ld_wait(r);
                tmem_ld_wait(q);
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    x[0][i] = __uint_as_float(r[i]);
                    x[1][i] = __uint_as_float(q[i]);
                }
            }
            if (!tma) {
                epilogue_turned_gated<T>(e, m0, n0 + c, p.Mp, p.Nq, lane, sa, x[0], x[1]);
                continue;
            }
            const float bias_n[2] = {bias_c[0], bias_c[1]}, sw_n[2] = {sw_c[0], sw_c[1]};
            fetch_columns(c + 64);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (e.sa) {
#pragma unroll
                    for (int i = 0; i < 32; i += 2)
                        split(mul(f2(x[h][i], x[h][i + 1]), f2(sa)), x[h][i], x[h][i + 1]);
                }
                if (e.sw) apply_columns<true>(sw_n[h], x[h]);
                if (e.bias) {
                    if constexpr (kBiasSmem) {
                        const uint4* v = reinterpret_cast<const uint4*>(bias_s + (c / 64 * 2 + h) * 32);
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            float f[8];
                            unpack8<T>(v[g], f);
#pragma unroll
                            for (int i = 0; i < 8; i += 2)
                                split(add(f2(x[h][8 * g + i], x[h][8 * g + i + 1]), f2(f[i], f[i + 1])),
                                      x[h][8 * g + i], x[h][8 * g + i + 1]);
                        }
                    } else {
                        apply_columns<false>(bias_n[h], x[h]);
                    }
                }
            }
            if (e.Z) {
                emit(mapZ, x[0], n0 + c, m0);
                emit(mapZu, x[1], n0 + c, m0);
            }
            act_n<T>(e.act, x[0]);
#pragma unroll
            for (int i = 0; i < 32; i += 2)
                split(mul(f2(x[0][i], x[0][i + 1]), f2(x[1][i], x[1][i + 1])), x[0][i], x[0][i + 1]);
            emit(mapY, x[0], n0 + c, m0);
            __syncwarp();
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&s.acc_empty[b]), 0u));
    }
    if (lane == 0) bulk_wait_group_read<0>();
}

template <typename T, bool GATED>
__global__ void __launch_bounds__(kTileThreads, 1)
    linear_tile_kernel(const __grid_constant__ CUtensorMap mapP, const __grid_constant__ CUtensorMap mapQ,
                       const __grid_constant__ CUtensorMap mapY, const __grid_constant__ CUtensorMap mapZ,
                       const __grid_constant__ CUtensorMap mapR, const __grid_constant__ TcLinear p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const TileSmem s = carve_tile(smem_raw, p);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = int(cluster_ctarank());
    const int cid = blockIdx.x / 2, ncl = gridDim.x / 2;
    const uint32_t stage_bytes = p.p_bytes + p.q_bytes;
    const uint64_t tmo = p.timeout_ns;
    if (warp == 0 && lane == 0) {
        prefetch_tensormap(&mapP);
        prefetch_tensormap(&mapQ);
        if (p.tma_out) {
            prefetch_tensormap(&mapY);
            if (p.e.Z) prefetch_tensormap(&mapZ);
            if (GATED ? p.e.Z != nullptr : p.e.R != nullptr) prefetch_tensormap(&mapR);
        }
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.acc_full[i], 1);
            mbar_init(&s.acc_empty[i], 2 * kTileEpiWarps);  // both CTAs' epilogue warps
        }
        mbar_init(s.drain, 1);
        for (int i = 0; i < 2 * kTileEpiWarps; ++i) mbar_init(&s.rbar[i], 1);
        s.abort[0] = s.abort[1] = 0;
        s.peer[2] = 0;
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
    int fills = 0;  // a producer's
    uint32_t rphase = 0, rpend = 0;  // residual fills: next parity, and in flight (bit: buffer)

    const int prod = warp == 0 ? 0 : (warp == 2 ? 1 : -1);
    if (prod >= 0) {
        const uint64_t pol = l2_policy(2);  // panels are read again by later tiles
        const int q_rows = p.bn / 2;        // of this CTA's half
        const int q_atoms = (q_rows + 63) / 64;
        const uint32_t tx = 2u * (p.p_bytes + (p.q_mn ? uint32_t(q_atoms) * kAtom : uint32_t(q_rows) * 128u));
        const uint32_t stages0 = smem_u32(s.stages), full0 = smem_u32(s.full);
        const uint32_t lead0 = mapa_shared(full0, 0);  // both CTAs' fills complete on the even one's
        const int nstages = p.stages, nk = p.k_blocks;
        int stage = 0, turn = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = cid; ok && t < p.tiles; t += ncl) {
            int tp, tq;
            tile_at(t, p, tp, tq);
            const int p0 = (2 * tp + rank) * 128;
            const int q0 = GATED ? tq * q_rows + rank * int(p.Nq) : tq * p.bn + rank * q_rows;
            int kb = p.k_rotate ? int(int64_t(t) * nk / p.tiles) : 0;
            if (t == cid) {
                grid_dependency_wait();
                s.abort[1] = 1;
            }
            for (int i = 0; i < nk; ++i, turn ^= 1, kb = kb + 1 == nk ? 0 : kb + 1) {
                if (turn == prod) {
                    if (!__all_sync(0xffffffffu, wait_bounded(&s.empty[stage], phase ^ 1u, s.abort, tmo))) {
                        ok = false;
                        break;
                    }
                    const uint32_t sp = stages0 + uint32_t(stage) * stage_bytes;
                    const uint32_t lead = lead0 + 8u * uint32_t(stage);
                    const int k0 = kb * p.bk;
                    if (rank == 0) expect_elected(full0 + 8u * uint32_t(stage), tx);
                    load_operand<true>(sp, &mapP, lead, p.p_mn, 2, p0, k0, pol);
                    load_operand<true>(sp + p.p_bytes, &mapQ, lead, p.q_mn, q_atoms, q0, k0, pol);
                    ++fills;
                }
                if (++stage == nstages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
    }
    if (warp == 1 && rank == 0) {
        const uint64_t dP = smem_desc_with_addr(operand_desc(p.p_mn), smem_u32(s.stages));
        const uint64_t dQ = smem_desc_with_addr(operand_desc(p.q_mn), smem_u32(s.stages) + p.p_bytes);
        const uint64_t step_p = operand_step(p.p_mn), step_q = operand_step(p.q_mn);
        const uint32_t idesc = p.idesc, stage_units = stage_bytes >> 4;
        const uint32_t empty0 = smem_u32(s.empty);
        const int nstages = p.stages, nk = p.k_blocks;
        const bool fp8 = p.fp8 != 0;
        int stage = 0, it = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int t = cid; ok && t < p.tiles; t += ncl, ++it) {
            const int b = it & 1;
            if (!__all_sync(0xffffffffu, wait_bounded(&s.acc_empty[b], ((it >> 1) & 1) ^ 1u, s.abort, tmo)))
                break;
            tc_fence_after_sync();
            const uint32_t acc = tmem + uint32_t(b) * 256u;
            for (int kb = 0; kb < nk; ++kb) {
                if (!__all_sync(0xffffffffu, wait_bounded(&s.full[stage], phase, s.abort, tmo))) {
                    ok = false;
                    break;
                }
                tc_fence_after_sync();
                const uint64_t off = uint64_t(uint32_t(stage) * stage_units);
                issue_stage<true>(fp8, acc, dP + off, dQ + off, step_p, step_q, idesc, kb != 0,
                                  empty0 + 8u * uint32_t(stage), 3);
                if (++stage == nstages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            if (ok) commit_elected_pair(&s.acc_full[b], 3);
        }
        commit_elected_pair(s.drain, 1);
        wait_bounded(s.drain, 0, s.abort, tmo, true);
    }
    if (GATED && warp >= 4) {
        grid_dependency_wait();
        gated_epilogue<T>(p, s, mapY, mapZ, mapR, tmem, warp, lane, rank, cid, ncl);
    }
    if (!GATED && warp >= 4) {
        grid_dependency_wait();
        const int ew = warp - 4, quad = warp & 3, half = ew >> 2;
        const uint32_t lanes = uint32_t(quad * 32) << 16;
        uint8_t* const staging = s.staging + ew * kStaging;
        uint64_t* const rbar = s.rbar + 2 * ew;
        constexpr int kBuf = 1024 * int(sizeof(T));           // one 32 x 32 tile
        constexpr int kBufs = kStaging / kBuf;                // 2, or 1 of 32-bit outputs
        const bool tma = p.tma_out != 0;
        const bool staged_z = tma && p.e.Z;
        const bool staged_r = tma && p.e.R && !p.e.Z;         // (with Z the buffers are taken)
        const uint64_t pol = l2_policy(1);                    // outputs pass through once
        int it = 0;
        // The buffer of the next chunk. Without Z and R it alternates on from one
        // tile to the next: each use waits for all stores but the latest, which
        // an odd number of chunks would otherwise leave in the first buffer.
        int j = 0;
        for (int t = cid; t < p.tiles; t += ncl, ++it) {
            int tp, tq;
            tile_at(t, p, tp, tq);
            const int64_t m0 = int64_t(2 * tp + rank) * 128 + quad * 32, m = m0 + lane;
            const int64_t q0 = int64_t(tq) * p.bn;
            const int b = it & 1;
            const bool live = m < p.Mp;
            // This warp's chunks: columns c = 32 half, + 64, ... below limit.
            const int limit = m0 < p.Mp ? int(max(int64_t(0), min(int64_t(p.bn), p.Nq - q0))) : 0;
            auto fetch_r = [&](int c, int buf) {  // lane 0; the buffer's last store has been read
                mbar_arrive_expect_tx(&rbar[buf], kBuf);
                tma_load_2d_hint(staging + buf * kBuf, &mapR, &rbar[buf], int(q0) + c, int(m0), pol);
            };
            if (staged_r) {
                j = 0;
                if (lane == 0) bulk_wait_group_read<0>();
                for (int i = 0; i < kBufs; ++i)
                    if (32 * half + 64 * i < limit) {
                        if (lane == 0) fetch_r(32 * half + 64 * i, i);
                        rpend |= 1u << i;
                    }
                __syncwarp();
            }
            const float sa = live && p.e.sa ? p.e.sa[m] : 1.f;
            // While the MMAs run: a 16-bit bias of the warp's columns into shared
            // memory, from where every lane reads all of it; a 32-bit bias and
            // the columns' scales into a register of the column's lane, a chunk
            // ahead, to be passed round by shuffles.
            constexpr bool kBiasSmem = sizeof(T) == 2;
            T* const bias_s = reinterpret_cast<T*>(s.bias + ew * kBiasBytes);
            float bias_c = 0.f, sw_c = 1.f;
            auto fetch_columns = [&](int c) {
                const int64_t n = q0 + c + lane;
                if (c < limit && n < p.Nq) {
                    if (!kBiasSmem && p.e.bias) bias_c = to_f32(static_cast<const T*>(p.e.bias)[n]);
                    if (p.e.sw) sw_c = p.e.sw[n];
                }
            };
            if (tma) {
                if (kBiasSmem && p.e.bias) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int64_t n = q0 + 32 * half + 64 * i + lane;
                        if (32 * half + 64 * i < limit && n < p.Nq)
                            bias_s[32 * i + lane] = static_cast<const T*>(p.e.bias)[n];
                    }
                    __syncwarp();
                }
                fetch_columns(32 * half);
            }
            bool ok = wait_bounded(&s.acc_full[b], (it >> 1) & 1, s.abort, tmo);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t acc = tmem + lanes + uint32_t(b * 256);
            for (int c = 32 * half; c < limit; c += 64, j ^= kBufs - 1) {
                float x[32];
                {
                    uint32_t r[32];
                    tmem_ld_32x32b_x32(acc + uint32_t(c), r);
                    tmem_ld_wait(r);
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(r[i]);
                }
                if (!tma) {
                    epilogue_turned<T>(p.e, m0, q0 + c, p.Mp, p.Nq, lane, sa, x);
                    continue;
                }
                const int64_t n = q0 + c;
                const float bias_n = bias_c, sw_n = sw_c;
                fetch_columns(c + 64);
                if (p.e.sa) {
#pragma unroll
                    for (int i = 0; i < 32; i += 2)
                        split(mul(f2(x[i], x[i + 1]), f2(sa)), x[i], x[i + 1]);
                }
                if (p.e.sw) apply_columns<true>(sw_n, x);
                if (p.e.bias) {
                    if constexpr (kBiasSmem) {
                        const uint4* v = reinterpret_cast<const uint4*>(bias_s + c / 64 * 32);
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            float f[8];
                            unpack8<T>(v[g], f);
#pragma unroll
                            for (int i = 0; i < 8; i += 2)
                                split(add(f2(x[8 * g + i], x[8 * g + i + 1]), f2(f[i], f[i + 1])),
                                      x[8 * g + i], x[8 * g + i + 1]);
                        }
                    } else {
                        apply_columns<false>(bias_n, x);
                    }
                }
                uint8_t* buf = staging + j * kBuf;
                if (staged_z) {
                    // Two 16-bit buffers: Z's and Y's; one 32-bit buffer in turn.
                    if (lane == 0) {
                        if (kBufs == 2) bulk_wait_group_read<1>();
                        else bulk_wait_group_read<0>();
                    }
                    __syncwarp();
                    stage_row32<T>(staging, lane, x);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d_hint(&mapZ, staging, int(n), int(m0), pol);
                        bulk_commit_group();
                    }
                    buf = staging + (kBufs - 1) * kBuf;
                }
                act_n<T>(p.e.act, x);
                if (staged_r) {
                    bool rok = wait_bounded(&rbar[j], (rphase >> j) & 1u, s.abort, tmo);
                    ok = __all_sync(0xffffffffu, rok);
                    if (!ok) break;
                    rphase ^= 1u << j;
                    rpend &= ~(1u << j);
                    add_staged32<T>(buf, lane, p.e.rest, x);
                } else {
                    if (p.e.R && live) {
#pragma unroll
                        for (int g = 0; g < 4; ++g) {
                            float f[8];
                            const int64_t left = p.Nq - (n + 8 * g);
                            load8<T>(p.e.R, m * p.e.ldr + n + 8 * g, left >= 8, left < 8 ? int(left) : 8, f);
                            add_residual<T>(p.e.rest, f, x + 8 * g);
                        }
                    }
                    // The buffer's last store has been read (with Z: all but Z's).
                    if (lane == 0) {
                        if (kBufs == 2) bulk_wait_group_read<1>();
                        else bulk_wait_group_read<0>();
                    }
                    __syncwarp();
                }
                stage_row32<T>(buf, lane, x);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    tma_store_2d_hint(&mapY, buf, int(n), int(m0), pol);
                    bulk_commit_group();
                }
                if (staged_r && c + 64 * kBufs < limit) {
                    if (lane == 0) {
                        bulk_wait_group_read<0>();
                        fetch_r(c + 64 * kBufs, j);
                    }
                    rpend |= 1u << j;
                }
                __syncwarp();
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&s.acc_empty[b]), 0u));
            if (!ok) break;
        }
        if (lane == 0) bulk_wait_group_read<0>();
        if (*s.abort)
            for (int i = 0; i < 2; ++i)
                if (rpend & (1u << i)) wait_bounded(&rbar[i], (rphase >> i) & 1u, s.abort, tmo, true);
    }
    tc_fence_before_sync();
    __syncthreads();
    const bool gave_up = *s.abort != 0;
    if (gave_up && prod >= 0 && lane == 0) {
        s.fills[prod] = fills;
        const uint32_t peer = mapa_shared(smem_u32(const_cast<int*>(s.peer)), uint32_t(rank ^ 1));
        st_cluster_b32(peer + 4u * uint32_t(prod), uint32_t(fills));
        if (prod == 0) st_cluster_b32(peer + 8u, 1u);
    }
    cluster_sync();  // no CTA leaves while a peer may still reach its barriers
    // (Where only one gave up, the other has seen all MMAs through and with them
    // all fills.)
    if (gave_up && s.peer[2]) {
        if (rank == 0 && threadIdx.x == 0) {
            const int q_rows = p.bn / 2;
            drain_fills(s, p, p.p_bytes + (p.q_mn ? uint32_t((q_rows + 63) / 64) * kAtom : uint32_t(q_rows) * 128u), tmo);
        }
        cluster_sync();
    }
    if (warp == 1) {
        __syncwarp();
        tc_fence_after_sync();
        tmem_dealloc<2>(tmem, 512);
    }
}

// ------------------------------------------------------------ split kernel
// 8 warps: 0 issues the TMA fills, 1 the MMAs and owns tensor memory, and all
// of them join and write the tile. A block that stays within half of an SM's
// shared memory shares the SM with another one, whose fills run under this
// one's set-up and joining.
//
// The tile's lines along the output's contiguous direction are dealt out to the
// cluster's CTAs in turn. Each CTA stores its partial sums of a line straight
// from tensor memory into the shared memory of the line's owner, over the
// stages once all CTAs' MMAs are done, or at once into room left beside them;
// after a cluster barrier the owners add up and write their lines, in rank
// order, so results repeat. What passes
// between SMs moves at 17 bytes a clock into each, by loads, stores or bulk
// copies alike (96 KB in a cluster of 4: 6860, 5730, 6030 clocks); stores need
// no round trip (144 x 4096 x 4096: 12.5 us against 13.4 with loads).
constexpr int kSplitThreads = 256;

struct SplitSmem {
    uint8_t* stages;  // then the partial sums
    uint64_t *full, *empty, *acc_full;
    uint32_t* tmem_base;
    volatile int* abort;  // and [1], see wait_bounded
};

__device__ __forceinline__ SplitSmem carve_split(uint8_t* raw, const TcLinear& p) {
    SplitSmem s;
    s.stages = raw;  // 1024-byte aligned
    uint64_t* bars = reinterpret_cast<uint64_t*>(raw + p.ring_bytes);
    s.full = bars;
    s.empty = bars + p.stages;
    s.acc_full = bars + 2 * p.stages;
    s.tmem_base = reinterpret_cast<uint32_t*>(s.acc_full + 1);
    s.abort = reinterpret_cast<volatile int*>(s.tmem_base + 1);
    return s;
}

// The two halves of cluster_sync().
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Four neighbouring outputs n.. of row m (cnt of them in the matrix; vec: all
// four, and every pointer's address there a multiple of four elements).
template <typename T>
__device__ __forceinline__ void load4(const void* base, int64_t at, bool vec, int cnt, float (&f)[4]) {
    const T* p = static_cast<const T*>(base) + at;
    if (vec) {
        if constexpr (sizeof(T) == 4) {
            const float4 v = *reinterpret_cast<const float4*>(p);
            f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
        } else {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            float g[8];
            unpack8<T>(make_uint4(v.x, v.y, 0, 0), g);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = g[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = i < cnt ? to_f32(p[i]) : 0.f;
    }
}

template <typename T>
__device__ __forceinline__ void store4(void* base, int64_t at, bool vec, int cnt, const float (&f)[4]) {
    T* p = static_cast<T*>(base) + at;
    if (vec) {
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
        } else {
            const float g[8] = {f[0], f[1], f[2], f[3], 0.f, 0.f, 0.f, 0.f};
            const uint4 v = pack8<T>(g);
            *reinterpret_cast<uint2*>(p) = make_uint2(v.x, v.y);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < cnt) p[i] = from_f32<T>(f[i]);
    }
}

// Line l of a tile is rank l % SPLIT's, the l / SPLIT-th of its lines; an owner
// holds `per` lines of every rank's partial sums, a rank's one after the other.
// This stores the accumulators of the first `rows` lines there.
template <int SPLIT, bool SWAP>
__device__ __forceinline__ void deal_lines(const TcLinear& p, uint32_t tmem, float* part, int per, int pitch,
                                           int rank, int rows) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = warp & 3, pl = quad * 32 + lane;
    const uint32_t mine = smem_u32(part) + uint32_t(rank * per * pitch) * 4u;
    for (int c = warp >> 2; 32 * c < p.bn; c += 2) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(tmem + (uint32_t(quad * 32) << 16) + uint32_t(32 * c), r);
        tmem_ld_wait(r);
        if (!SWAP && SPLIT == 1) {  // a lane is a line
            if (pl < rows)
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    if (32 * c + i < p.bn)
                        *reinterpret_cast<uint4*>(part + pl * pitch + 32 * c + i) =
                            make_uint4(r[i], r[i + 1], r[i + 2], r[i + 3]);
        } else {  // a lane is a place in each of 32 lines, so that stores are contiguous
            if (!SWAP) transpose32(lane, r);
            const int place = SWAP ? pl : 32 * c + lane;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int l = (SWAP ? 32 * c : 32 * quad) + i;
                if (l < rows && (SWAP || place < p.bn)) {
                    if (SPLIT == 1)
                        part[l * pitch + place] = __uint_as_float(r[i]);
                    else
                        st_cluster_b32(mapa_shared(mine + uint32_t(l / SPLIT * pitch + place) * 4u,
                                                   uint32_t(i % SPLIT)), r[i]);
                }
            }
        }
        __syncwarp();
    }
}

// Adds up and writes this CTA's lines, of `cols` values: a line to a warp at a
// time, four values to a lane, kAhead lines' sums in flight. Bias and column
// scales are the same for all lines and loaded once.
template <typename T, int SPLIT>
__device__ __forceinline__ void join_lines(const TcLinear& p, const float* part, int per, int pitch, int rank,
                                           int rows, int cols, int64_t m0, int64_t n0) {
    constexpr int kAhead = SPLIT == 8 ? 2 : 4;
    constexpr int kWarps = kSplitThreads / 32;
    const Epilogue& e = p.e;
    const int owned = (rows - rank + SPLIT - 1) / SPLIT;
    const int first = int(threadIdx.x >> 5);
    for (int at = 4 * int(threadIdx.x & 31); at < cols; at += 128) {
        const int cnt = min(4, cols - at);
        const bool vec = p.vec && cnt == 4;
        const int64_t n = n0 + at;
        float bias[4] = {}, sw[4] = {1.f, 1.f, 1.f, 1.f};
        if (e.bias) load4<T>(e.bias, n, vec, cnt, bias);
        if (e.sw) load4<float>(e.sw, n, vec, cnt, sw);
        for (int line = first; line < owned; line += kWarps * kAhead) {
            float x[kAhead][4];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                // (Past the last line: the last one again, not written.)
                const float* own = part + min(line + j * kWarps, owned - 1) * pitch + at;
                float4 v[SPLIT];
#pragma unroll
                for (int r = 0; r < SPLIT; ++r) v[r] = *reinterpret_cast<const float4*>(own + r * per * pitch);
                x[j][0] = v[0].x;
                x[j][1] = v[0].y;
                x[j][2] = v[0].z;
                x[j][3] = v[0].w;
#pragma unroll
                for (int r = 1; r < SPLIT; ++r) {
                    x[j][0] += v[r].x;
                    x[j][1] += v[r].y;
                    x[j][2] += v[r].z;
                    x[j][3] += v[r].w;
                }
            }
            float res[kAhead][4];
            if (e.R) {
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {
                    const int64_t m = m0 + min(line + j * kWarps, owned - 1) * SPLIT + rank;
                    load4<T>(e.R, m * e.ldr + n, vec, cnt, res[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (line + j * kWarps >= owned) break;
                const int64_t m = m0 + (line + j * kWarps) * SPLIT + rank;
                const float sa = e.sa ? e.sa[m] : 1.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) x[j][i] = fmaf(x[j][i], sa * sw[i], bias[i]);
                if (e.Z) store4<T>(e.Z, m * e.ldz + n, vec, cnt, x[j]);
                act_n<T>(e.act, x[j]);
                if (e.R) add_residual<T>(e.rest, res[j], x[j]);
                store4<T>(e.Y, m * e.ldy + n, vec, cnt, x[j]);
            }
        }
    }
}

// The same of the gated layer: a line's values are `half` gates and as many
// factors, `cols` of each in the matrix. Lines are short, so a warp takes several
// at a time, 16 or 32 lanes to each.
template <typename T, int SPLIT>
__device__ __forceinline__ void join_gated(const TcLinear& p, const float* part, int per, int pitch, int rank,
                                           int rows, int cols, int half, int64_t N, int64_t m0, int64_t n0) {
    const Epilogue& e = p.e;
    const int owned = (rows - rank + SPLIT - 1) / SPLIT;
    const int side = half <= 64 ? 16 : 32;  // lanes to a line
    for (int at = 4 * int(threadIdx.x % side); at < cols; at += 4 * side) {
        const int cnt = min(4, cols - at);
        const bool vec = p.vec && cnt == 4;
        const int64_t n = n0 + at;
        float bias[2][4] = {}, sw[2][4] = {{1.f, 1.f, 1.f, 1.f}, {1.f, 1.f, 1.f, 1.f}};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (e.bias) load4<T>(e.bias, n + h * N, vec, cnt, bias[h]);
            if (e.sw) load4<float>(e.sw, n + h * N, vec, cnt, sw[h]);
        }
        for (int line = int(threadIdx.x) / side; line < owned; line += kSplitThreads / side) {
            const float* own = part + line * pitch + at;
            const int64_t m = m0 + line * SPLIT + rank;
            float4 v[2][SPLIT];
#pragma unroll
            for (int r = 0; r < SPLIT; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    v[h][r] = *reinterpret_cast<const float4*>(own + r * per * pitch + h * half);
            const float sa = e.sa ? e.sa[m] : 1.f;
            float x[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                x[h][0] = v[h][0].x;
                x[h][1] = v[h][0].y;
                x[h][2] = v[h][0].z;
                x[h][3] = v[h][0].w;
#pragma unroll
                for (int r = 1; r < SPLIT; ++r) {
                    x[h][0] += v[h][r].x;
                    x[h][1] += v[h][r].y;
                    x[h][2] += v[h][r].z;
                    x[h][3] += v[h][r].w;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) x[h][i] = fmaf(x[h][i], sa * sw[h][i], bias[h][i]);
                if (e.Z) store4<T>(e.Z, m * e.ldz + n + h * N, vec, cnt, x[h]);
            }
            act_n<T>(e.act, x[0]);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[0][i] *= x[1][i];
            store4<T>(e.Y, m * e.ldy + n, vec, cnt, x[0]);
        }
    }
}

template <typename T, bool SWAP, bool GATED>
__global__ void __launch_bounds__(kSplitThreads, 2)
    linear_split_kernel(const __grid_constant__ CUtensorMap mapP, const __grid_constant__ CUtensorMap mapQ,
                        const __grid_constant__ TcLinear p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const SplitSmem s = carve_split(smem_raw, p);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = int(cluster_ctarank());
    const int tile = blockIdx.x / p.split;
    const int tp = tile % p.tiles_p, tq = tile / p.tiles_p;
    // (Gated weights come as two boxes, each of half the rows, the second one's
    // `up` rows after the first's.)
    const int p0 = GATED && SWAP ? tp * (p.bp / 2) : tp * p.bp, q0 = GATED && !SWAP ? tq * (p.bn / 2) : tq * p.bn;
    const int up = GATED ? int(SWAP ? p.Mp : p.Nq) : 0;
    const int kb0 = int(int64_t(p.k_blocks) * rank / p.split);
    const int kb1 = int(int64_t(p.k_blocks) * (rank + 1) / p.split);
    const int nk = kb1 - kb0;
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
        s.abort[0] = s.abort[1] = 0;
        fence_mbarrier_init();
    }
    if (warp == 1) {
        tmem_alloc<1>(s.tmem_base, uint32_t(p.tmem_cols));
        tmem_relinquish_alloc_permit<1>();
    }
    tc_fence_before_sync();
    __syncthreads();
    if (p.split > 1 && p.sums_at != 0) cluster_arrive();
    tc_fence_after_sync();
    grid_launch_dependents();
    const uint32_t tmem = *s.tmem_base;
    uint32_t issued_any = 0, issued_parity = 0;
    if (warp == 0) {
        const uint64_t pol_p = l2_policy(p.tiles_q == 1 ? 1 : 2), pol_q = l2_policy(2);
        const int q_atoms = (p.bn + 63) / 64, p_atoms = (p.bp + 63) / 64;
        const uint32_t tx = (p.p_mn ? uint32_t(p_atoms) * kAtom : uint32_t(p.bp) * 128u) +
                            (p.q_mn ? uint32_t(q_atoms) * kAtom : uint32_t(p.bn) * 128u);
        const uint32_t stages0 = smem_u32(s.stages), full0 = smem_u32(s.full);
        const int nstages = p.stages;
        // Ask L2 for the first stages' boxes before waiting for the previous
        // grid: its writes land in L2 too, so no line there is ever stale.
        for (int i = 0; i < nk && i < nstages; ++i) {
            const int k0 = (kb0 + i) * p.bk;
            if (p.p_mn) {
                for (int a = 0; a < p_atoms; ++a) prefetch_elected(&mapP, p0 + 64 * a, k0);
            } else {
                prefetch_elected(&mapP, k0, p0);
                if (GATED && SWAP) prefetch_elected(&mapP, k0, p0 + up);
            }
        }
        grid_dependency_wait();
        s.abort[1] = 1;
        int stage = 0;
        uint32_t phase = 0;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!__all_sync(0xffffffffu, wait_bounded(&s.empty[stage], phase ^ 1u, s.abort, tmo))) break;
            const uint32_t sp = stages0 + uint32_t(stage) * stage_bytes, bar = full0 + 8u * uint32_t(stage);
            const int k0 = kb * p.bk;
            expect_elected(bar, tx);
            load_operand<false>(sp, &mapP, bar, p.p_mn, p_atoms, p0, k0, pol_p);
            load_operand<false>(sp + p.p_bytes, &mapQ, bar, p.q_mn, q_atoms, q0, k0, pol_q);
            if (GATED && SWAP) load_elected<false>(sp + uint32_t(p.bp) * 64u, &mapP, bar, k0, p0 + up, pol_p);
            if (GATED && !SWAP)
                load_elected<false>(sp + p.p_bytes + uint32_t(p.bn) * 64u, &mapQ, bar, k0, q0 + up, pol_q);
            issued_any |= 1u << stage;
            issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
            if (++stage == nstages) {
                stage = 0;
                phase ^= 1u;
            }
        }
    } else if (warp == 1) {
        const uint64_t dP = smem_desc_with_addr(operand_desc(p.p_mn), smem_u32(s.stages));
        const uint64_t dQ = smem_desc_with_addr(operand_desc(p.q_mn), smem_u32(s.stages) + p.p_bytes);
        const uint64_t step_p = operand_step(p.p_mn), step_q = operand_step(p.q_mn);
        const uint32_t idesc = p.idesc, stage_units = stage_bytes >> 4;
        const uint32_t empty0 = smem_u32(s.empty);
        const int nstages = p.stages;
        const bool fp8 = p.fp8 != 0;
        int stage = 0;
        uint32_t phase = 0;
        for (int i = 0; i < nk; ++i) {
            if (!__all_sync(0xffffffffu, wait_bounded(&s.full[stage], phase, s.abort, tmo))) break;
            tc_fence_after_sync();
            const uint64_t off = uint64_t(uint32_t(stage) * stage_units);
            issue_stage<false>(fp8, tmem, dP + off, dQ + off, step_p, step_q, idesc, i != 0,
                               empty0 + 8u * uint32_t(stage), 0);
            if (++stage == nstages) {
                stage = 0;
                phase ^= 1u;
            }
        }
        // Complete once every MMA issued is (also after a wait gave up).
        commit_elected(s.acc_full);
    }
    __syncwarp();
    // Every warp waits for the MMAs before it may read tensor memory, reuse the
    // stages or leave.
    bool ok = wait_bounded(s.acc_full, 0, s.abort, tmo, true);
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after_sync();
    float* part = reinterpret_cast<float*>(s.stages + p.sums_at);
    // Lines of bp (swapped) or bn values, four words more apart.
    const int pitch = (SWAP ? 128 : p.bn) + 4;
    const int64_t M = SWAP ? p.Nq : p.Mp, N = SWAP ? p.Mp : p.Nq;
    const int64_t m0 = SWAP ? q0 : p0, n0 = SWAP ? p0 : q0;
    const int width = (SWAP ? p.bp : p.bn) / (GATED ? 2 : 1);
    const int cols = int(min(int64_t(width), N - n0));
    const int rows = int(min(int64_t(SWAP ? p.bn : p.bp), M - m0));
    const auto deal_and_join = [&](auto n) {
        constexpr int kSplit = decltype(n)::value;
        const int per = (SWAP ? p.bn : p.bp) / kSplit;
        if (kSplit > 1) {
            // Peers have begun; without sums_at, their stages are idle too.
            if (p.sums_at == 0) cluster_arrive();
            cluster_wait();
        }
        if (__all_sync(0xffffffffu, ok && !*s.abort)) deal_lines<kSplit, SWAP>(p, tmem, part, per, pitch, rank, rows);
        tc_fence_before_sync();
        __syncwarp();
        if (kSplit > 1) cluster_sync();
        else __syncthreads();
        grid_dependency_wait();
        if (!*s.abort) {
            if constexpr (GATED) join_gated<T, kSplit>(p, part, per, pitch, rank, rows, cols, width, N, m0, n0);
            else join_lines<T, kSplit>(p, part, per, pitch, rank, rows, cols, m0, n0);
        }
    };
    switch (p.split) {
        case 1: deal_and_join(std::integral_constant<int, 1>()); break;
        case 2: deal_and_join(std::integral_constant<int, 2>()); break;
        case 4: deal_and_join(std::integral_constant<int, 4>()); break;
        default: deal_and_join(std::integral_constant<int, 8>()); break;
    }
    if (*s.abort && warp == 0 && lane == 0)
        for (int i = 0; i < p.stages; ++i)
            if (issued_any & (1u << i))
                wait_bounded(&s.full[i], (issued_parity >> i) & 1u, s.abort, tmo, true);
    __syncwarp();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc<1>(tmem, uint32_t(p.tmem_cols));
    }
}

using TileFn = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, TcLinear);
using SplitFn = void (*)(CUtensorMap, CUtensorMap, TcLinear);

template <typename T>
TileFn pick_tile_typed(const TcLinear& p) {
    return p.gated ? linear_tile_kernel<T, true> : linear_tile_kernel<T, false>;
}

TileFn pick_tile(const TcLinear& p) {
    return p.e.out == TPGEMM_ELEM_F16    ? pick_tile_typed<__half>(p)
           : p.e.out == TPGEMM_ELEM_BF16 ? pick_tile_typed<__nv_bfloat16>(p)
                                         : pick_tile_typed<float>(p);
}

template <typename T>
SplitFn pick_split_typed(const TcLinear& p) {
    if (p.gated) return p.swap ? linear_split_kernel<T, true, true> : linear_split_kernel<T, false, true>;
    return p.swap ? linear_split_kernel<T, true, false> : linear_split_kernel<T, false, false>;
}

SplitFn pick_split(const TcLinear& p) {
    return p.e.out == TPGEMM_ELEM_F16    ? pick_split_typed<__half>(p)
           : p.e.out == TPGEMM_ELEM_BF16 ? pick_split_typed<__nv_bfloat16>(p)
                                         : pick_split_typed<float>(p);
}

int cluster_of(const TcLinear& p) { return p.pair ? 2 : p.split; }

void set_cluster(cudaLaunchAttribute& a, int n) {
    a.id = cudaLaunchAttributeClusterDimension;
    a.val.clusterDim.x = unsigned(n);
    a.val.clusterDim.y = 1;
    a.val.clusterDim.z = 1;
}

}  // namespace

size_t tc_linear_smem(const TcLinear& p) {
    if (p.pair)
        return size_t(p.stages) * (p.p_bytes + p.q_bytes) + kTileEpiWarps * (kStaging + kBiasBytes) +
               8 * (2 * size_t(p.stages) + 5 + 2 * kTileEpiWarps) + 32;
    return p.half_sm ? kSplitHalfSmem : size_t(kTcMaxSmem);
}

namespace {
// Lets a kernel use all shared memory.
cudaError_t allow_smem(const void* fn) {
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kTcMaxSmem);
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(fn, cudaFuncAttributePreferredSharedMemoryCarveout,
                                 cudaSharedmemCarveoutMaxShared);
    return e;
}
}  // namespace

cudaError_t launch_tc_linear(const TcLinearMaps& maps, const TcLinear& p, int grid, cudaStream_t stream) {
    const int cluster = cluster_of(p);
    const size_t ring = size_t(p.stages) * (p.p_bytes + p.q_bytes);
    if (p.stages < 2 || p.stages > 32 || cluster < 1 || cluster > 8 || grid % cluster != 0 ||
        p.bn % 16 != 0 || p.bn > 256 || (p.pair && (p.bn % 32 != 0 || p.group < 1)) ||
        (p.gated && (p.pair ? p.bn % 64 != 0 : (p.swap ? p.p_mn : p.q_mn) != 0)) ||
        (!p.pair && (p.bp > 128 || p.bp % 16 != 0 || p.split > p.k_blocks || (p.split & (p.split - 1)) ||
                     ring > (p.sums_at ? p.sums_at : p.ring_bytes) ||
                     split_partial_bytes(p) + p.sums_at > p.ring_bytes ||
                     p.ring_bytes + 8 * (2 * size_t(p.stages) + 1) + 16 > tc_linear_smem(p))))
        return cudaErrorInvalidValue;
    const size_t smem = tc_linear_smem(p);
    if (smem > size_t(kTcMaxSmem)) return cudaErrorInvalidConfiguration;
    const TileFn tile = pick_tile(p);
    const SplitFn split = pick_split(p);
    cudaError_t e = allow_smem(p.pair ? reinterpret_cast<const void*>(tile) : reinterpret_cast<const void*>(split));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(p.pair ? kTileThreads : kSplitThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    set_cluster(attr[1], cluster);
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if (p.pair) return cudaLaunchKernelEx(&cfg, tile, maps.P, maps.Q, maps.Y, maps.Z, maps.R, p);
    return cudaLaunchKernelEx(&cfg, split, maps.P, maps.Q, p);
}

cudaError_t tc_linear_max_pairs(const TcLinear& p, int* pairs) {
    const TileFn fn = pick_tile(p);
    cudaError_t e = allow_smem(reinterpret_cast<const void*>(fn));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kTileThreads);
    cfg.dynamicSmemBytes = tc_linear_smem(p);
    cudaLaunchAttribute attr[1];
    set_cluster(attr[0], 2);
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
