// Host-side interfaces of the operators around the multiply (linear layer, its
// gradients, root-mean-square norm and its gradients) between their entry
// points (ops_api.cu) and their kernels. Not part of the public ABI.
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
// Y, Z, R and bias are of type `out`; every pointer but Y may be null.
struct Epilogue {
    void* Y;
    void* Z;
    const void* R;
    const void* bias;
    const float* sa;
    const float* sw;
    int64_t ldy, ldz, ldr;
    int act, out;
};

// Y = epilogue(A B^T): A has M rows, B has N rows, both K columns of `dtype`.
struct LinearOp {
    int64_t M, N, K;
    int dtype;
    Operand a, b;
    Epilogue e;
};

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

}  // namespace tpg
