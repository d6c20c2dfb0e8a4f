// The tcgen05 kernels of the linear layer: their parameters and launch.
#pragma once

#include "ops_internal.h"

namespace tpg {

struct TcLinear {
    Epilogue e;
    int64_t Mp, Nq;        // rows of P and of Q (gated: half of the weights')
    int gated;             // see LinearOp: a tile's weight rows are of both halves
    uint64_t timeout_ns;   // bound of every wait
    int tiles_p, tiles_q;  // a cluster's tiles along P and Q
    int tiles;             // tile kernel: their number
    int k_blocks, bk;      // 128-byte-wide K stages, and K elements of each
    int bp, bn;            // P rows of a split tile; Q rows of a tile
    int p_mn, q_mn;        // operand stored along its rows
    int stages;            // depth of the TMA ring
    uint32_t p_bytes, q_bytes;  // shared bytes of one stage's operands (of one CTA)
    uint32_t ring_bytes;   // split kernel: shared bytes of ring and partial sums
    uint32_t sums_at;      // split kernel: their place; 0: over the stages
    uint32_t idesc;
    int tmem_cols;         // split kernel
    int split;             // split kernel: CTAs of a cluster, each a share of K
    int group;             // tile kernel: P tiles in a raster run
    int k_rotate;          // tile kernel: tiles start at different places of K
    int half_sm;           // split kernel: half of an SM's shared memory, two blocks to an SM
    int tma_out;           // tile kernel: Y, Z and R move by TMA (rows of whole units on 16-byte boundaries)
    int swap;              // P holds the output's columns
    int pair;              // tile kernel (1) or split kernel (0)
    int fp8;
    int vec;               // split kernel: four outputs move as one access
};

struct TcLinearMaps {
    CUtensorMap P, Q;     // operands
    CUtensorMap Y, Z, R;  // tile kernel with tma_out: 32 x 32 boxes (gated: Z's halves)
};

size_t tc_linear_smem(const TcLinear& p);
cudaError_t launch_tc_linear(const TcLinearMaps& maps, const TcLinear& p, int grid, cudaStream_t stream);
// CTA pairs of the tile kernel that fit the device at once.
cudaError_t tc_linear_max_pairs(const TcLinear& p, int* pairs);
// Shared memory of a split block that leaves room for another on its SM.
constexpr size_t kSplitHalfSmem = 112 * 1024;
// Shared bytes of a split tile's partial sums.
inline size_t split_partial_bytes(const TcLinear& p) {
    return p.swap ? size_t(p.bn) * (128 + 4) * 4 : size_t(p.bp) * (p.bn + 4) * 4;
}
constexpr size_t kTileStagingBytes = 8 * (4096 + 256);  // of the epilogue's warps
cudaError_t linear_read_and_clear_status(int* status);

}  // namespace tpg
