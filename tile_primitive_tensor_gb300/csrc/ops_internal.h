// Host-side interfaces of the operators around the multiply (linear layer, its
// gradients, norms and their gradients, dropout) between their entry points
// (ops_api.cu) and their kernels. Not part of the public ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "tpgemm.h"

namespace tpg {

// From tpgemm_api.cu: records the calling thread's error reason and returns s
// (printf format); the current device's checks (compute capability 10.3); the
// driver's tensor-map encoder.
tpgemm_status fail_with(tpgemm_status s, const char* fmt, ...);
tpgemm_status require_device(int* sms);
tpgemm_status tensor_map_encoder(PFN_cuTensorMapEncodeTiled_v12000* fn);

// Planner overrides of the linear layer's product (TPGEMM_LINEAR_PATH, _BN, _BP,
// _SPLIT; -1: not set), from the snapshot that tpgemm_reload_tuning renews.
enum { kLinearTile = 0, kLinearSplit = 1, kLinearFew = 2 };
struct LinearTuning {
    int path, bn, bp, split;
};
LinearTuning linear_tuning();

// Streaming multiprocessors of a GB300. Grids and plans of these operators are
// sized by it. It is a constant, not the device's count, since the strips of
// column sums go by it too: results and workspaces are then the same everywhere.
constexpr int kSms = 152;

// Terms that tensor memory adds up in one go for a 32-bit result of the gated layer:
// its additions truncate, so a sum is off by some 1.2e-9 of its size for each term.
constexpr int64_t kLongSum = 4096;

inline int elem_size(int elem) {
    return elem == TPGEMM_ELEM_F32 ? 4 : (elem == TPGEMM_ELEM_F16 || elem == TPGEMM_ELEM_BF16) ? 2 : 1;
}

// ---- the linear layer's product ----
// An operand of `rows` rows and K columns: element (r, k) is p[r ld + k], or
// p[k ld + r] when it is stored along its rows (mn).
struct Operand {
    const void* p;
    int64_t ld;
    int mn;
};

// What happens to an accumulator x of output (m, n):
//   z = sa[m] sw[n] x + bias[n]  (z is stored to Z when given),
//   Y[m, n] = act(z) + R[m, n].
// Y, Z, R and bias are of type `out`; every pointer but Y may be null. rest: z is what
// R, a 32-bit sum of the same terms' larger parts, lacks, and is left out where R is not
// finite (an infinity times the parts may be a NaN where it is an infinity times the
// whole).
struct Epilogue {
    void* Y;
    void* Z;
    const void* R;
    const void* bias;
    const float* sa;
    const float* sw;
    int64_t ldy, ldz, ldr;
    int act, out;
    int rest = 0;
};

// Y = epilogue(A B^T): A has M rows, B has N rows, both K columns of `dtype`.
// Gated: B has 2 N rows, sw, bias and Z as many columns; of an output's two
// accumulators the first gives the gate z (B's row n), the second the factor u
// (row N + n), both stored to Z, and Y[m, n] = act(z) u. R is null then.
struct LinearOp {
    int64_t M, N, K;
    int dtype;
    Operand a, b;
    Epilogue e;
    int gated = 0;
};
// Rows of B.
inline int64_t weight_rows(const LinearOp& op) { return op.gated ? 2 * op.N : op.N; }

// The product on the tcgen05 kernels (linear_plan.cu); its operands' rows start
// on 16-byte boundaries (tma_rows). K >= 1.
tpgemm_status run_linear_tc(const LinearOp& op, int sms, cudaStream_t stream);

// The product for few rows of A (linear_few.cu), operands K-contiguous, any
// alignment, any K.
constexpr int kFewTokens = 16;
bool linear_few_takes(const LinearOp& op);
bool linear_few_wins(const LinearOp& op);
// Whether every line of the operand starts on a 128-byte boundary.
bool whole_lines(const Operand& o, int64_t rows, int64_t K, int dtype);
cudaError_t launch_linear_few(const LinearOp& op, int sms, cudaStream_t stream);

bool tma_rows(const Operand& o, int64_t rows, int64_t K, int dtype);

// ---- gradients of the linear layer's epilogue ----
// dZ = dY act'(Z) (dZ is not written when act is none) and per-strip column
// sums of dZ, then their sum over the strips into dbias.
struct ActGradOp {
    int64_t M, N;
    const void* dY;
    const void* Z;
    int64_t lddy, ldz;
    void* dZ;         // [M][lddz], or null
    int64_t lddz;
    float* partial;   // [strips][N] for dbias of more than one strip
    void* dbias;      // or null
    int dtype, act, grad;
};
int act_grad_strips(int64_t M, int64_t N);
cudaError_t launch_act_grad(const ActGradOp& op, cudaStream_t stream);

// The gated layer's: dZ [M][2 N] from dY [M][N] and Z [M][2 N], dbias [2 N],
// partial [strips][2 N].
int gated_grad_strips(int64_t M, int64_t N);
// What dZ lost to its rounding: low [M][lddz] = (dZ - its rounding) / scale[n], with
// scale [2 N] a power of two; or null.
struct DzRest {
    void* low;
    float* scale;
};
cudaError_t launch_gated_grad(const ActGradOp& op, const DzRest& rest, cudaStream_t stream);

// Copies of matrices, each of rows of `bytes` bytes, `pitch` bytes apart, to rows
// dst_pitch apart (dst and dst_pitch multiples of 16, dst_pitch >= bytes rounded
// up to 16); one launch for all of them, none for none.
struct AlignJob {
    const uint8_t* src;
    int64_t rows, bytes, pitch;
    uint8_t* dst;
    int64_t dst_pitch;
};
struct AlignJobs {
    AlignJob j[3];
    int n;
};
cudaError_t launch_align_rows(const AlignJobs& jobs, cudaStream_t stream);

// ---- root-mean-square norm ----
struct RmsNormOp {
    int64_t rows, cols;
    const void* X;
    const void* R;      // or null
    const void* gamma;
    void* H;            // or null
    void* Y;
    void* scale;        // float [rows] (row) or E8M0 [rows][ceil(cols / 32)] (MX)
    float* rstd;        // or null
    int64_t ldx, ldr, ldh, ldy;
    int x, g, y;        // element types
    int mode;           // tpgemm_scale_mode
    float eps;
};
cudaError_t launch_rmsnorm(const RmsNormOp& op, cudaStream_t stream);

struct RmsNormGradOp {
    int64_t rows, cols;
    const void* dY;
    const void* H;
    const float* rstd;
    const void* gamma;
    const void* dH;     // or null
    void* dX;           // or null
    void* dgamma;       // or null
    float* partial;     // [strips][cols] when dgamma is given
    int64_t lddy, ldh, lddh, lddx;
    int x, g, grad;
};
int rmsnorm_grad_strips(int64_t rows, int64_t cols);
cudaError_t launch_rmsnorm_grad(const RmsNormGradOp& op, cudaStream_t stream);

// ---- dropout ----
// Element (i, j) is kept when its random word is at least `threshold` (the
// probability to drop it times 2^32), and multiplied by `scale`.
struct Drop {
    uint32_t key[10][2];      // of each round, from the seed (drop_keys)
    uint64_t offset;
    const uint64_t* counter;  // in device memory, added to offset; or null
    uint32_t threshold;
    float scale;
    int on;  // 0: nothing is dropped, and nothing above is read
};

inline void drop_keys(Drop* d, uint64_t seed) {
    for (uint32_t i = 0; i < 10; ++i) {
        d->key[i][0] = uint32_t(seed) + i * 0x9E3779B9u;
        d->key[i][1] = uint32_t(seed >> 32) + i * 0xBB67AE85u;
    }
}

struct DropoutOp {
    int64_t rows, cols;
    const void* X;
    const void* R;  // or null
    void* Y;
    int64_t ldx, ldr, ldy;
    int elem;
    Drop drop;
};
cudaError_t launch_dropout(const DropoutOp& op, cudaStream_t stream);

// ---- layer norm ----
struct LayerNormOp {
    int64_t rows, cols;
    const void* X;
    const void* R;      // or null
    const void* gamma;
    const void* beta;   // or null
    void* H;            // or null
    void* Y;
    float* scale;       // [rows] with TPGEMM_SCALE_ROW
    float* mean;        // or null
    float* rstd;        // or null
    int64_t ldx, ldr, ldh, ldy;
    int x, g, y;        // element types
    int mode;           // TPGEMM_SCALE_NONE or _ROW
    float eps;
    Drop drop;
};
cudaError_t launch_layernorm(const LayerNormOp& op, cudaStream_t stream);

struct LayerNormGradOp {
    int64_t rows, cols;
    const void* dY;
    const void* H;
    const float* mean;
    const float* rstd;
    const void* gamma;
    const void* dH;     // or null
    void* dX;           // or null
    void* dR;           // or null
    void* dgamma;       // or null
    void* dbeta;        // or null
    float* partial;     // [strips][2][cols], or null when neither is wanted
    int64_t lddy, ldh, lddh, lddx, lddr;
    int x, g, grad;
    Drop drop;
};
int layernorm_grad_strips(int64_t rows, int64_t cols);  // (at most)
cudaError_t launch_layernorm_grad(const LayerNormGradOp& op, cudaStream_t stream);

}  // namespace tpg
