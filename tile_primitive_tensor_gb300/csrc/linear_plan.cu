// Planning of the linear layer's product on the tcgen05 kernels: which kernel,
// orientation, tile and split, the tensor maps, and the launch.
#include <algorithm>
#include <mutex>

#include "linear_tc.h"
#include "ptx.cuh"
#include "tpgemm_internal.h"

namespace tpg {
namespace {

constexpr int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// CTA pairs of the tile kernel that fit the device at once, asked once per
// device (all variants hold the same threads and nearly all shared memory).
tpgemm_status max_pairs(const TcLinear& p, int* pairs) {
    static std::mutex m;
    static int cache[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) return fail_with(TPGEMM_ERR_ARCH, "device index %d unsupported", dev);
    std::lock_guard<std::mutex> lock(m);
    int& n = cache[dev];
    if (!n) {
        const cudaError_t e = tc_linear_max_pairs(p, &n);
        if (e != cudaSuccess || n <= 0) {
            n = 0;
            return fail_with(TPGEMM_ERR_LAUNCH, "cluster occupancy query failed: %s",
                             cudaGetErrorString(e));
        }
    }
    *pairs = n;
    return TPGEMM_OK;
}

// The models below are in ns at the clocks that products run at here (1.85
// GHz): an SM takes in 64 bytes a clock from memory or L2, and 17 from other
// SMs; memory delivers about 5.5 kB a ns to all SMs together, L2 about 13 to
// CTAs that each read a P tile of their own.
constexpr double kClock = 1.85;
constexpr double kMemory = 5500;
constexpr double kL2 = 13000;
constexpr double kPeer = 17;

// Shared bytes of one split stage. P tiles of fewer than 128 rows leave the MMA
// to read on into the bytes behind them: their lanes' results are not used.
uint32_t split_p_bytes(int bp, bool mn) { return mn ? uint32_t((bp + 63) / 64) * 8192u : uint32_t(bp) * 128u; }
uint32_t split_q_bytes(int bn, bool mn) { return mn ? uint32_t((bn + 63) / 64) * 8192u : uint32_t(bn) * 128u; }

// Stages of a split CTA in `have` bytes of shared memory (16 KB behind the last
// P tile's start are read at most).
int split_stages(size_t have, uint32_t p_bytes, uint32_t q_bytes) {
    const size_t over = 16384 > p_bytes + q_bytes ? 16384 - (p_bytes + q_bytes) : 0;
    return int(std::min<size_t>(12, (have - over) / (p_bytes + q_bytes)));
}

constexpr size_t kBarrierBytes = 512;

struct Choice {
    double ns = 1e30;
    int pair = 0, swap = 0, bn = 0, bp = 128, split = 1, half_sm = 0;
};

}  // namespace

bool tma_rows(const Operand& o, int64_t rows, int64_t K, int dtype) {
    const int64_t lines = o.mn ? K : rows;
    return reinterpret_cast<uintptr_t>(o.p) % 16 == 0 &&
           (lines <= 1 || (o.ld * elem_size(dtype)) % 16 == 0);
}

bool whole_lines(const Operand& o, int64_t rows, int64_t K, int dtype) {
    const int64_t lines = o.mn ? K : rows;
    return reinterpret_cast<uintptr_t>(o.p) % 128 == 0 && (lines <= 1 || (o.ld * elem_size(dtype)) % 128 == 0);
}

namespace {

// box_rows: rows of a K-contiguous box; K rows of a box along the operand's rows.
tpgemm_status encode(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, const Operand& o,
                     int64_t rows, int64_t K, int dtype, int box_rows) {
    const int es = elem_size(dtype);
    const CUtensorMapDataType t = es == 1                      ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                  : dtype == TPGEMM_ELEM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                              : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    const uint64_t inner = uint64_t(o.mn ? rows : K), outer = uint64_t(o.mn ? K : rows);
    cuuint64_t dims[2] = {inner, outer};
    // (A single line's pitch is never used, but has to be a multiple of 16.)
    cuuint64_t pitch[1] = {outer > 1 ? uint64_t(o.ld) * es : (inner * es + 15) / 16 * 16};
    cuuint32_t box[2] = {cuuint32_t(128 / es), cuuint32_t(box_rows)};
    cuuint32_t one[2] = {1, 1};
    const CUresult r = enc(map, t, 2, const_cast<void*>(o.p), dims, pitch, box, one,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail_with(TPGEMM_ERR_LAUNCH, "cuTensorMapEncodeTiled failed with CUresult %d", int(r));
    return TPGEMM_OK;
}

// Y, Z or R: 32 x 32 boxes, staged in shared memory with the swizzle of their
// 64- or 128-byte rows.
tpgemm_status encode_out(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, const void* base,
                         int64_t M, int64_t N, int64_t ld, int elem) {
    const int es = elem_size(elem);
    const CUtensorMapDataType t = es == 4                    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                  : elem == TPGEMM_ELEM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                             : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    cuuint64_t dims[2] = {uint64_t(N), uint64_t(M)};
    cuuint64_t pitch[1] = {M > 1 ? uint64_t(ld) * es : (uint64_t(N) * es + 15) / 16 * 16};
    cuuint32_t box[2] = {32, 32}, one[2] = {1, 1};
    const CUresult r = enc(map, t, 2, const_cast<void*>(base), dims, pitch, box, one,
                           CU_TENSOR_MAP_INTERLEAVE_NONE,
                           es == 4 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        return fail_with(TPGEMM_ERR_LAUNCH, "cuTensorMapEncodeTiled failed with CUresult %d", int(r));
    return TPGEMM_OK;
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Whether every row of Y, Z and R starts on a 16-byte boundary.
bool tma_outputs(const Epilogue& e, int64_t M) {
    const int es = elem_size(e.out);
    auto rows16 = [&](const void* p, int64_t ld) {
        return !p || (aligned16(p) && (M <= 1 || (ld * es) % 16 == 0));
    };
    return rows16(e.Y, e.ldy) && rows16(e.Z, e.ldz) && rows16(e.R, e.ldr);
}

// Whether rows of N values are whole units of 16 bytes, which is what a TMA store writes:
// of a row that ends inside one, the rest of that unit is written too (with zeros), though
// it lies outside of the tensor map. Such rows are turned and stored by element (2048 x
// 4093 bf16 with a stride of 4096, K = 1024: 23.6 us, all 4096 columns 14.9).
bool whole_units(int64_t N, int elem) { return N * elem_size(elem) % 16 == 0; }

// Costs and plans are of the accumulators: of a gated product's op N is taken as
// twice its own, which is also how many tiles of bn / 2 (bp / 2) outputs it has.
double memory_ns(const LinearOp& op) {
    return double((op.M + op.N) * op.K * elem_size(op.dtype) + 2 * op.M * op.N) / kMemory;
}

// The tile kernel: waves of 256 x bn tiles. A K stage is bound by what an SM
// takes in (128 + bn / 2 rows of 128 bytes; 7 % over that measured), which at
// bn = 256 is the tensor rate too, and takes 225 ns at the least (512 x 4096 x
// 4096 bf16: 20.3 us at bn = 128, 24.0 at 256; 4096^3: 74.8 at 224, 78.8 at 256).
// Short sums are bound by the epilogue, which has a fixed part to a tile (4096 x
// 4096 x 64 f16: 16.5 us at 256, 19.4 at 128, 28.4 at 64).
// Q's rows off the 128-byte lines take a seventh longer (144 x 16384 x 4096 f16
// 28.6 -> 32.5 us; P's 28.8).
Choice plan_tile(const LinearOp& op, int64_t kb, int sms, const LinearTuning& t) {
    Choice best;
    const double memory = memory_ns(op);
    const double off_lines = whole_lines(op.b, op.N, op.K, op.dtype) ? 1.0 : 1.15;
    for (int bn = 256; bn >= 32; bn -= 32) {
        if (t.bn > 0 && bn != t.bn) continue;
        if (op.gated && bn % 64) continue;  // halves of whole 32-column chunks
        const int64_t tiles = ceil_div(op.M, 256) * ceil_div(op.N, bn);
        const double stage = std::max(225.0, (256 + bn) * (bn == 256 ? 1.01 : 1.07) / kClock) * off_lines;
        const double mmas = double(kb) * stage + 200, epilogue = 1300 + 6.7 * bn;
        const double loop = std::max(mmas + double(ceil_div(tiles, sms / 2) - 1) * std::max(mmas, epilogue), memory);
        const double ns = 3500 + bn * 18 + loop;
        if (ns < best.ns) {
            best.ns = ns;
            best.pair = 1;
            best.bn = bn;
        }
    }
    return best;
}

// Blocks that run at once in clusters of `split`, placed within groups of SMs: 76
// of 2, 36 of 4 and 15 of 8 blocks that have an SM each, as the occupancy query
// counted them. Chips differ in which SMs a group has, by a cluster or two; a plan
// that counts on too many runs a few of its clusters late, with the same result.
int64_t places(int split, bool half_sm) {
    return (split <= 2 ? kSms : split == 4 ? 144 : 120) * (half_sm ? 2 : 1);
}

// What L2 costs the split kernel more when a row's stages of Q, which many
// tiles read, do not start on 128-byte lines and take two of them (144 x 16384
// x 4096 f16, split 1: 27.6 us, 32.9 with Q off the lines, 39.6 with P too, 27.8
// with P alone).
double straddle(const LinearOp& op, bool swap) {
    const bool a = whole_lines(op.a, op.M, op.K, op.dtype), b = whole_lines(op.b, op.N, op.K, op.dtype);
    if (swap ? a : b) return 1.0;
    return a || b ? 1.25 : 1.5;
}

// The split kernel with Q in tiles_q tiles. Blocks take half of an SM's shared
// memory while that holds five stages, and are then two to an SM; the tile's
// height and the split are those that fill the most of those places, 128 rows
// counting a fifth more, since shorter boxes stream more slowly (17 x 4096 x
// 4096 bf16, split / rows: 8 / 128 8.1 us, 4 / 128 8.5, 2 / 64 13.9; 144 rows:
// 4 / 128 12.3, 2 / 64 15.4).
Choice plan_split(const LinearOp& op, int64_t kb, const LinearTuning& t, int64_t tiles_q, int least) {
    Choice best;
    // The output's longer side along the lanes; Q in tiles of equal width.
    const bool swap = op.N >= op.M;
    const int64_t Mp = swap ? op.N : op.M, Nq = swap ? op.M : op.N;
    const bool p_mn = swap ? op.b.mn : op.a.mn, q_mn = swap ? op.a.mn : op.b.mn;
    TcLinear p{};
    p.swap = swap;
    p.bn = int(ceil_div(ceil_div(Nq, tiles_q), 16) * 16);
    tiles_q = ceil_div(Nq, p.bn);
    double most = -1;
    for (int bp = 128; bp >= 64; bp -= 16) {
        if (t.bp > 0 ? bp != t.bp : bp == 80) continue;
        if (p_mn && bp % 64) continue;
        p.bp = bp;
        const uint32_t p_bytes = split_p_bytes(bp, p_mn), q_bytes = split_q_bytes(p.bn, q_mn);
        const size_t half = kSplitHalfSmem - kBarrierBytes;
        const int half_sm = split_partial_bytes(p) <= half && split_stages(half, p_bytes, q_bytes) >= 5;
        const int64_t tiles = ceil_div(Mp, bp) * tiles_q;
        int split = 1;
        while (split < 8 && tiles * split * 2 <= places(split * 2, half_sm) && split * 4 <= kb) split *= 2;
        if (t.split == 1 || t.split == 2 || t.split == 4 || t.split == 8)
            for (split = t.split; split > kb; split /= 2) {
            }
        split = std::max(split, least);
        const int64_t ctas = tiles * split;
        const int64_t fit = places(split, half_sm);
        const double filled = double(std::min(ctas, fit)) / double(places(1, half_sm)) * (bp == 128 ? 1.2 : 1.0);
        if (filled <= most) continue;
        most = filled;
        best.swap = swap;
        best.bn = p.bn;
        best.bp = bp;
        best.split = split;
        best.half_sm = half_sm;
        const double share = double(ceil_div(kb, split)), resident = double(ceil_div(ctas, kSms));
        const double busy = resident * share * 2.0 * (bp + p.bn) / kClock;
        const double l2 = double(ctas) * share * (bp + p.bn) * 128 * straddle(op, swap) / kL2;
        const double sums = resident * bp * p.bn * 4;  // bytes an SM joins
        const double join = split > 1 ? 1000 + sums * (split - 1) / split / kPeer / kClock : sums / 128;
        best.ns = 4300.0 * double(ceil_div(ctas, fit)) + join + std::max(busy, std::max(memory_ns(op), l2));
    }
    return best;
}

// The number of Q tiles: one more of them makes the tiles narrower and the
// split shallower, so that less passes between SMs but P is read more often
// (512 x 1024 x 4096 bf16, tiles of Q / split: 2 / 4 15.3 us, 3 / 4 12.4, 4 / 4
// 11.5; 144 x 4096 x 4096: 1 / 4 12.5, 2 / 2 14.8).
Choice plan_split(const LinearOp& op, int64_t kb, const LinearTuning& t, int least_split) {
    const int64_t Nq = std::min(op.M, op.N), least = ceil_div(Nq, 256);
    Choice best;
    for (int64_t q = least; q < least + 4 && q * 32 <= std::max(Nq, least * 32); ++q) {
        const Choice c = plan_split(op, kb, t, q, least_split);
        if (c.ns < best.ns) best = c;
    }
    return best;
}

// A gated 32-bit output is a product of two sums, and off by both of theirs: sums
// of more than kLongSum terms are shared out to CTAs, whose shorter ones are added
// with rounding (2048 x 2048 outputs of random signs, K = 16384 in four shares:
// 8.2e-6 of their size). Eight shares are the most: they keep to kLongSum up to K =
// 32768, and past it grow with K. The tile kernel, whatever its cost or the override of
// the path, does not take these products: it adds all of K in one piece.
int least_split(const LinearOp& op) {
    int split = 1;
    if (op.gated && op.e.out == TPGEMM_ELEM_F32)
        while (split < 8 && op.K > split * kLongSum) split *= 2;
    return split;
}

}  // namespace

tpgemm_status run_linear_tc(const LinearOp& op, int sms, cudaStream_t stream) {
    PFN_cuTensorMapEncodeTiled_v12000 enc;
    tpgemm_status s = tensor_map_encoder(&enc);
    if (s != TPGEMM_OK) return s;
    const LinearTuning t = linear_tuning();
    TcLinear p{};
    p.e = op.e;
    p.fp8 = elem_size(op.dtype) == 1;
    p.bk = p.fp8 ? 128 : 64;
    p.k_blocks = int(ceil_div(op.K, p.bk));
    p.timeout_ns = wait_timeout_ns();
    LinearOp wide = op;  // (see memory_ns)
    wide.N = weight_rows(op);
    const int least = least_split(op);
    const Choice split = plan_split(wide, p.k_blocks, t, least);
    Choice c = plan_tile(wide, p.k_blocks, sms, t);
    if (t.path == kLinearSplit || least > 1 || (t.path != kLinearTile && split.ns < c.ns)) c = split;
    if (c.bn == 0) return fail_with(TPGEMM_ERR_PATH, "the planner overrides leave no plan");
    p.pair = c.pair;
    p.swap = c.swap;
    p.bn = c.bn;
    p.bp = c.bp;
    p.split = c.split;
    p.half_sm = c.half_sm;
    p.gated = op.gated;
    // (The gated layer's second halves of Z, bias and scales start N elements on.)
    const bool halves = !op.gated || whole_units(op.N, op.e.out);
    p.tma_out = p.pair && tma_outputs(op.e, op.M) && whole_units(op.N, op.e.out);
    p.vec = !p.pair && tma_outputs(op.e, op.M) && aligned16(op.e.bias) && aligned16(op.e.sw) && halves;
    const Operand& P = p.swap ? op.b : op.a;
    const Operand& Q = p.swap ? op.a : op.b;
    p.Mp = p.swap ? op.N : op.M;
    p.Nq = p.swap ? op.M : op.N;
    p.p_mn = P.mn;
    p.q_mn = Q.mn;
    p.idesc = idesc_f16_f32(op.dtype == TPGEMM_ELEM_BF16 || op.dtype == TPGEMM_ELEM_E5M2, P.mn != 0,
                            Q.mn != 0, p.pair ? 256 : 128, p.bn);
    const int q_rows = p.pair ? p.bn / 2 : p.bn;
    p.p_bytes = p.pair ? 16384u : split_p_bytes(p.bp, P.mn != 0);
    p.q_bytes = split_q_bytes(q_rows, Q.mn != 0);
    const int64_t rows_p = p.swap ? wide.N : p.Mp, rows_q = p.swap ? p.Nq : wide.N;
    const int64_t tiles_p = ceil_div(rows_p, p.pair ? 256 : p.bp);
    const int64_t tiles_q = ceil_div(rows_q, p.bn);
    if (tiles_p * tiles_q * p.split > 0x1fffffff)
        return fail_with(TPGEMM_ERR_SHAPE, "too many tiles");
    p.tiles_p = int(tiles_p);
    p.tiles_q = int(tiles_q);
    p.tiles = int(tiles_p * tiles_q);
    const size_t budget = size_t(kTcMaxSmem) - kBarrierBytes;
    int grid;
    if (p.pair) {
        p.stages = int(std::min<size_t>(8, (budget - kTileStagingBytes) / (p.p_bytes + p.q_bytes)));
        p.group = 8;
        // Few tiles along one side: the CTAs at work all read the same panels.
        p.k_rotate = p.tiles_p == 1 || p.tiles_q == 1;
        int pairs = 0;
        s = max_pairs(p, &pairs);
        if (s != TPGEMM_OK) return s;
        grid = 2 * std::min(p.tiles, pairs);
    } else {
        const size_t have = p.half_sm ? kSplitHalfSmem - kBarrierBytes : budget;
        const uint32_t stage = p.p_bytes + p.q_bytes, sums = uint32_t((split_partial_bytes(p) + 1023) / 1024 * 1024);
        p.stages = split_stages(have, p.p_bytes, p.q_bytes);
        // A split that needs few stages leaves room for the sums beside them.
        const int few = std::max(2, int(ceil_div(p.k_blocks, p.split)));
        const uint32_t few_bytes = std::max(uint32_t(few) * stage, uint32_t(few - 1) * stage + 16384u);
        if (p.split > 1 && few <= p.stages && few_bytes + sums <= have) {
            p.stages = few;
            p.sums_at = (few_bytes + 1023u) / 1024u * 1024u;
            p.ring_bytes = p.sums_at + sums;
        } else {
            p.ring_bytes = std::max(std::max(uint32_t(p.stages) * stage, sums), uint32_t(p.stages - 1) * stage + 16384u);
        }
        p.tmem_cols = 32;
        while (p.tmem_cols < 32 * ((p.bn + 31) / 32)) p.tmem_cols *= 2;
        grid = p.tiles * p.split;
    }
    TcLinearMaps maps;
    // (Gated weights come as two boxes, but to the pairs, whose CTAs load half each.)
    s = encode(enc, &maps.P, P, rows_p, op.K, op.dtype,
               P.mn ? 64 : p.pair ? 128 : op.gated && p.swap ? p.bp / 2 : p.bp);
    if (s != TPGEMM_OK) return s;
    s = encode(enc, &maps.Q, Q, rows_q, op.K, op.dtype,
               Q.mn ? 64 : op.gated && !p.pair && !p.swap ? q_rows / 2 : q_rows);
    if (s != TPGEMM_OK) return s;
    maps.Y = maps.Z = maps.R = maps.P;
    if (p.tma_out) {
        const Epilogue& o = op.e;
        s = encode_out(enc, &maps.Y, o.Y, op.M, op.N, o.ldy, o.out);
        if (s == TPGEMM_OK && o.Z) s = encode_out(enc, &maps.Z, o.Z, op.M, op.N, o.ldz, o.out);
        if (s == TPGEMM_OK && o.Z && op.gated)
            s = encode_out(enc, &maps.R, static_cast<const uint8_t*>(o.Z) + op.N * elem_size(o.out), op.M, op.N,
                           o.ldz, o.out);
        if (s == TPGEMM_OK && o.R) s = encode_out(enc, &maps.R, o.R, op.M, op.N, o.ldr, o.out);
        if (s != TPGEMM_OK) return s;
    }
    const cudaError_t e = launch_tc_linear(maps, p, grid, stream);
    if (e != cudaSuccess)
        return fail_with(TPGEMM_ERR_LAUNCH, "tcgen05 linear kernel launch: %s", cudaGetErrorString(e));
    return TPGEMM_OK;
}

}  // namespace tpg
