// Dropout's random words: Philox4x32 of ten rounds (Salmon, Moraes, Dror and
// Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011). The words of
// element (i, j) are a function of the seed, the offset, i and j alone:
//   counter (j / 4, i, offset low, offset high), key (seed low, seed high),
//   word j % 4, kept when word >= round(p 2^32),
// so no mask is stored, the backward pass draws the same one again, and the
// result hangs neither on strides nor on how threads share the work.
//
// A counter gives four elements 128 bits for twenty 32 x 32 -> 64-bit products,
// five to an element, which a multiprocessor does at half the rate of additions.
#pragma once

#include "vec8.cuh"

namespace tpg {
namespace {

struct DropKey {
    uint32_t k0, k1, o0, o1, threshold;
    float scale;
};

// (Reads the counter in memory: after the grid dependency.)
__device__ __forceinline__ DropKey drop_key(const Drop& d) {
    uint64_t offset = d.offset;
    if (d.counter) offset += *d.counter;
    return {uint32_t(d.seed), uint32_t(d.seed >> 32), uint32_t(offset), uint32_t(offset >> 32), d.threshold,
            d.scale};
}

__device__ __forceinline__ uint4 philox(const DropKey& k, uint32_t row, uint32_t block) {
    uint32_t c0 = block, c1 = row, c2 = k.o0, c3 = k.o1;
#pragma unroll
    for (uint32_t i = 0; i < 10; ++i) {
        const uint64_t a = uint64_t(c0) * 0xD2511F53u, b = uint64_t(c2) * 0xCD9E8D57u;
        c0 = uint32_t(b >> 32) ^ c1 ^ (k.k0 + i * 0x9E3779B9u);
        c1 = uint32_t(b);
        c2 = uint32_t(a >> 32) ^ c3 ^ (k.k1 + i * 0xBB67AE85u);
        c3 = uint32_t(a);
    }
    return make_uint4(c0, c1, c2, c3);
}

// A dropped element is 0 whatever it held, a kept one x / (1 - p).
__device__ __forceinline__ float drop_one(const DropKey& k, uint32_t word, float x) {
    return word >= k.threshold ? x * k.scale : 0.f;
}

// Four neighbouring elements from column 4 * block on.
__device__ __forceinline__ void drop4(const DropKey& k, uint32_t row, uint32_t block, float* x) {
    const uint4 w = philox(k, row, block);
    x[0] = drop_one(k, w.x, x[0]);
    x[1] = drop_one(k, w.y, x[1]);
    x[2] = drop_one(k, w.z, x[2]);
    x[3] = drop_one(k, w.w, x[3]);
}

// Eight elements of a lane, element j at column first + j step, first % 4 equal
// to lane % 4 and step a multiple of 4: four lanes need the four words of one
// counter, so each of them draws those of every fourth j and they trade. The
// whole warp calls this.
__device__ __forceinline__ void drop8_apart(const DropKey& k, uint32_t row, int64_t first, int64_t step,
                                            float (&x)[8]) {
    const int r = threadIdx.x & 3;
#pragma unroll
    for (int h = 0; h < 8; h += 4) {
        const uint4 w = philox(k, row, uint32_t((first + int64_t(h + r) * step) / 4));
        // Lane r gets word r of the counter that lane r ^ s drew, that of element h + (r ^ s).
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int want = r ^ s;
            const uint32_t give = want == 0 ? w.x : want == 1 ? w.y : want == 2 ? w.z : w.w;
            const uint32_t word = __shfl_xor_sync(0xffffffffu, give, s);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j == want) x[h + j] = drop_one(k, word, x[h + j]);
        }
    }
}

}  // namespace
}  // namespace tpg
