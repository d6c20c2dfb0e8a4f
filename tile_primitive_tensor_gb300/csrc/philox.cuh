// Dropout's random words: Philox4x32 of ten rounds (Salmon, Moraes, Dror and
// Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011). The words of
// element (i, j) are a function of the seed, the offset, i and j alone:
//   counter (j / 4, i, offset low, offset high), key (seed low, seed high),
//   word j % 4, kept when word >= round(p 2^32),
// so no mask is stored, the backward pass draws the same one again, and the
// result hangs neither on strides nor on how threads share the work.
//
// A counter gives four elements 128 bits for ten rounds of two 32 x 32 -> 64-bit
// products and two three-way exclusive ors. The rounds' keys lie with the kernel's
// parameters, from where the exclusive ors take them as operands; of the first two
// rounds one product each is the same along a row and is taken once. Products are what
// bounds it: a round takes a warp 8.5 cycles of its scheduler's quarter of an SM with
// their halves taken apart, 10.9 as one 64-bit product.
#pragma once

#include "vec8.cuh"

namespace tpg {
namespace {

// The offset's words, from which a row's draws start; what else a kernel needs it
// reads from its parameters.
struct DropOffset {
    uint32_t lo, hi;
};

// (Reads the counter in memory: after the grid dependency.)
__device__ __forceinline__ DropOffset drop_offset(const Drop& d) {
    uint64_t offset = d.offset;
    if (d.counter) offset += *d.counter;
    return {uint32_t(offset), uint32_t(offset >> 32)};
}

// What a row's counters share after the products that hang on the row alone.
struct DropRow {
    uint32_t r1, r3;  // round 1: its second word, and what its third is besides a product
    uint32_t p0, p1;  // round 2: the high and low half of the first word's product
};

__device__ __forceinline__ DropRow drop_row(const Drop& d, const DropOffset& o, uint32_t row) {
    const uint64_t b = uint64_t(o.lo) * 0xCD9E8D57u;
    const uint32_t c0 = uint32_t(b >> 32) ^ row ^ d.key[0][0];
    const uint64_t a = uint64_t(c0) * 0xD2511F53u;
    return {uint32_t(b), o.hi ^ d.key[0][1], uint32_t(a >> 32), uint32_t(a)};
}

// The words of the counter of columns 4 block .. 4 block + 3.
__device__ __forceinline__ uint4 philox(const Drop& d, const DropRow& r, uint32_t block) {
    constexpr uint32_t kA = 0xD2511F53u, kB = 0xCD9E8D57u;
    uint32_t c2 = __umulhi(block, kA) ^ r.r3, c3 = block * kA;                    // round 1
    uint32_t c0 = __umulhi(c2, kB) ^ r.r1 ^ d.key[1][0], c1 = c2 * kB;            // round 2
    c2 = r.p0 ^ c3 ^ d.key[1][1];
    c3 = r.p1;
#pragma unroll
    for (int i = 2; i < 10; ++i) {
        const uint32_t a = c0, b = c2;
        c0 = __umulhi(b, kB) ^ c1 ^ d.key[i][0];
        c1 = b * kB;
        c2 = __umulhi(a, kA) ^ c3 ^ d.key[i][1];
        c3 = a * kA;
    }
    return make_uint4(c0, c1, c2, c3);
}

// A dropped element is 0 whatever it held; a kept one is still to be multiplied
// by 1 / (1 - p), which a residual's addition takes along.
__device__ __forceinline__ float keep_one(const Drop& d, uint32_t word, float x) {
    return word >= d.threshold ? x : 0.f;
}

// Four neighbouring elements from column 4 * block on.
__device__ __forceinline__ void keep4(const Drop& d, const DropRow& r, uint32_t block, float* x) {
    const uint4 w = philox(d, r, block);
    x[0] = keep_one(d, w.x, x[0]);
    x[1] = keep_one(d, w.y, x[1]);
    x[2] = keep_one(d, w.z, x[2]);
    x[3] = keep_one(d, w.w, x[3]);
}

// Eight elements of a lane, element j at column first + j step, first % 4 equal
// to lane % 4 and step a multiple of 4: four lanes need the four words of one
// counter, so each of them draws those of every fourth j and they trade. The
// whole warp calls this.
__device__ __forceinline__ void keep8_apart(const Drop& d, const DropRow& row, int64_t first, int64_t step,
                                            float (&x)[8]) {
    const int r = threadIdx.x & 3;
#pragma unroll
    for (int h = 0; h < 8; h += 4) {
        const uint4 w = philox(d, row, uint32_t((first + int64_t(h + r) * step) / 4));
        // Lane r gets word r of the counter that lane r ^ s drew, that of element h + (r ^ s).
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int want = r ^ s;
            const uint32_t give = want == 0 ? w.x : want == 1 ? w.y : want == 2 ? w.z : w.w;
            const uint32_t word = __shfl_xor_sync(0xffffffffu, give, s);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j == want) x[h + j] = keep_one(d, word, x[h + j]);
        }
    }
}

}  // namespace
}  // namespace tpg
