// C-ABI entry points of the operators around the multiply: argument checks,
// the choice of kernels, and their launches on the caller's stream.
#include <algorithm>
#include <cmath>

#include "ops_internal.h"
#include "tpgemm_internal.h"

namespace {

using tpg::elem_size;
using tpg::fail_with;

bool is_16bit(int t) { return t == TPGEMM_ELEM_F16 || t == TPGEMM_ELEM_BF16; }
bool is_fp8(int t) { return t == TPGEMM_ELEM_E4M3 || t == TPGEMM_ELEM_E5M2; }
bool is_float(int t) { return is_16bit(t) || t == TPGEMM_ELEM_F32; }

size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

// A matrix argument: rows x cols elements of `elem`, rows `ld` elements apart.
struct Mat {
    const char* name;
    const void* p;
    int64_t rows, cols, ld;
    int elem;
    int64_t row_bytes() const { return cols * elem_size(elem); }
    int64_t pitch() const { return ld * elem_size(elem); }
    int64_t span() const { return rows > 0 ? (rows - 1) * pitch() + row_bytes() : 0; }
};

Mat vec(const char* name, const void* p, int64_t n, int elem) { return {name, p, 1, n, n, elem}; }

// Whether two matrices share a byte. Rows of one pitch interleave without
// touching when their positions within the pitch are disjoint (slices of one
// buffer); with different pitches any overlap of the spans counts.
bool share(const Mat& a, const Mat& b) {
    if (!a.p || !b.p || a.span() <= 0 || b.span() <= 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    if (x >= y + uintptr_t(b.span()) || y >= x + uintptr_t(a.span())) return false;
    if (a.rows > 1 && b.rows > 1 && a.pitch() != b.pitch()) return true;
    const int64_t pitch = a.rows > 1 ? a.pitch() : (b.rows > 1 ? b.pitch() : 0);
    if (pitch == 0) return true;
    const int64_t at = ((int64_t(y - x) % pitch) + pitch) % pitch;  // b's place in a's pitch
    return at < a.row_bytes() || pitch - at < b.row_bytes();
}

bool same(const Mat& a, const Mat& b) {
    return a.p && a.p == b.p && (a.rows <= 1 || a.pitch() == b.pitch()) && a.elem == b.elem;
}

constexpr int64_t kMaxDim = int64_t(1) << 30;

tpgemm_status check_dim(const char* name, int64_t v, int64_t least) {
    if (v < least || v >= kMaxDim)
        return fail_with(TPGEMM_ERR_SHAPE, "%s=%lld must be at least %lld and below 2^30", name,
                         (long long)v, (long long)least);
    return TPGEMM_OK;
}

// Presence, element alignment and row stride of one argument.
tpgemm_status check_mat(Mat& m, bool needed) {
    if (m.rows <= 0 || m.cols <= 0) return TPGEMM_OK;
    if (!m.p) return needed ? fail_with(TPGEMM_ERR_NULL, "%s is NULL", m.name) : TPGEMM_OK;
    if (reinterpret_cast<uintptr_t>(m.p) % uintptr_t(elem_size(m.elem)))
        return fail_with(TPGEMM_ERR_ALIGN, "%s=%p is not aligned to its %d-byte elements", m.name,
                         m.p, elem_size(m.elem));
    if (m.ld < m.cols || m.ld > (int64_t(1) << 40))
        return fail_with(TPGEMM_ERR_SHAPE, "%s: row stride %lld for %lld columns", m.name,
                         (long long)m.ld, (long long)m.cols);
    // (Not as a product: 2^30 rows of 2^42 bytes are past 64 bits.)
    if (m.pitch() / 16 + 1 > (int64_t(1) << 36) / m.rows)
        return fail_with(TPGEMM_ERR_SHAPE, "%s exceeds one GPU's memory", m.name);
    return TPGEMM_OK;
}

// No output shares bytes with an input or another output, but for the pairs in
// `in_place` (output index, input index) when they are the very same matrix.
struct Pair {
    int out, in;
};
tpgemm_status check_overlap(const Mat* out, int nout, const Mat* in, int nin, const Pair* in_place,
                            int npairs) {
    for (int i = 0; i < nout; ++i) {
        for (int j = i + 1; j < nout; ++j)
            if (share(out[i], out[j]))
                return fail_with(TPGEMM_ERR_ALIAS, "%s overlaps %s", out[i].name, out[j].name);
        for (int j = 0; j < nin; ++j) {
            if (!share(out[i], in[j])) continue;
            bool ok = false;
            for (int k = 0; k < npairs; ++k)
                ok = ok || (in_place[k].out == i && in_place[k].in == j && same(out[i], in[j]));
            if (!ok) return fail_with(TPGEMM_ERR_ALIAS, "%s overlaps %s", out[i].name, in[j].name);
        }
    }
    return TPGEMM_OK;
}

int64_t dense(int64_t ld, int64_t cols) { return ld == 0 ? cols : ld; }

tpgemm_status check_workspace(const void* ws, size_t have, size_t need, const Mat* mats, int n) {
    if (need == 0) return TPGEMM_OK;
    if (!ws) return fail_with(TPGEMM_ERR_NULL, "workspace is NULL; %zu bytes needed", need);
    if (reinterpret_cast<uintptr_t>(ws) % 256)
        return fail_with(TPGEMM_ERR_ALIGN, "workspace=%p is not 256-byte aligned", ws);
    if (have < need)
        return fail_with(TPGEMM_ERR_NULL, "workspace of %zu bytes; %zu needed", have, need);
    const Mat w{"workspace", ws, 1, int64_t(need), int64_t(need), TPGEMM_ELEM_E4M3};
    for (int i = 0; i < n; ++i) {
        // (Any byte between an operand's rows counts too.)
        const Mat span{mats[i].name, mats[i].p, 1, mats[i].span(), mats[i].span(), TPGEMM_ELEM_E4M3};
        if (share(w, span))
            return fail_with(TPGEMM_ERR_ALIAS, "the workspace overlaps %s", mats[i].name);
    }
    return TPGEMM_OK;
}

tpgemm_status launched(cudaError_t e, const char* what) {
    if (e != cudaSuccess)
        return fail_with(TPGEMM_ERR_LAUNCH, "%s: %s", what, cudaGetErrorString(e));
    return TPGEMM_OK;
}

tpgemm_status check_act(int act) {
    if (act < TPGEMM_ACT_NONE || act > TPGEMM_ACT_GELU_TANH)
        return fail_with(TPGEMM_ERR_DTYPE, "activation %d is not one of tpgemm_act", act);
    return TPGEMM_OK;
}

#define TPG_TRY(expr)                       \
    do {                                    \
        const tpgemm_status s_ = (expr);    \
        if (s_ != TPGEMM_OK) return s_;     \
    } while (0)

// Aligned copies of a product's operands in a workspace. An operand whose rows
// do not start on 16-byte boundaries cannot be read by TMA: it is copied to
// rows that do, which moves its bytes twice more (37 x 1000 x 1001 f16: 7.7 us
// with the copies, 6.0 at 40 x 1000 x 1000, which needs none). Copies start
// their rows on 128-byte lines.
struct Aligned {
    size_t at = 0;      // byte offset in the workspace
    int64_t ld = 0;     // row stride of the copy, elements
    bool copy = false;
};

Aligned plan_aligned(const tpg::Operand& o, int64_t rows, int64_t K, int dtype, size_t* total,
                     bool lines128 = false) {
    Aligned a;
    a.copy = !tpg::tma_rows(o, rows, K, dtype) || (lines128 && !tpg::whole_lines(o, rows, K, dtype));
    if (!a.copy) return a;
    const int64_t lines = o.mn ? K : rows, len = o.mn ? rows : K;
    const size_t es = size_t(elem_size(dtype));
    a.ld = int64_t(align_up(size_t(len) * es, 128) / es);
    a.at = *total;
    *total = align_up(*total + size_t(lines) * size_t(a.ld) * es, 256);
    return a;
}

// Points the operand at its place in the workspace and adds the copy to jobs.
void use_aligned(const Aligned& a, tpg::Operand* o, int64_t rows, int64_t K, int dtype, uint8_t* ws,
                 tpg::AlignJobs* jobs) {
    if (!a.copy) return;
    const int64_t lines = o->mn ? K : rows, len = o->mn ? rows : K;
    const int64_t es = elem_size(dtype);
    jobs->j[jobs->n++] = {static_cast<const uint8_t*>(o->p), lines, len * es, o->ld * es,
                          ws + a.at, a.ld * es};
    o->p = ws + a.at;
    o->ld = a.ld;
}

// Which product kernel takes it: the few-token one, or the tcgen05 ones. Few
// tokens on aligned rows run faster on tcgen05 once the weights are large.
bool takes_few(const tpg::LinearOp& op) {
    if (op.K == 0) return true;
    if (!tpg::linear_few_takes(op)) return false;
    const int path = tpg::linear_tuning().path;
    if (path >= 0) return path == tpg::kLinearFew;
    return tpg::linear_few_wins(op);
}

// One product; its operands are aligned unless the few-token kernel takes it.
tpgemm_status run_product(const tpg::LinearOp& op, int sms, cudaStream_t st) {
    if (takes_few(op))
        return launched(tpg::launch_linear_few(op, sms, st), "linear kernel launch");
    return tpg::run_linear_tc(op, sms, st);
}

// (The gated layer's 2 N rows of W are within the bound of sizes too.)
tpgemm_status check_linear_desc(const tpgemm_linear_desc* d, bool gated = false) {
    if (!d) return fail_with(TPGEMM_ERR_NULL, "the description is NULL");
    TPG_TRY(check_dim("M", d->M, 0));
    TPG_TRY(check_dim("N", d->N, 0));
    TPG_TRY(check_dim("K", d->K, 0));
    if (gated) TPG_TRY(check_dim("2 N", 2 * d->N, 0));
    if (!is_16bit(d->dtype) && !is_fp8(d->dtype))
        return fail_with(TPGEMM_ERR_DTYPE, "A and W must be f16, bf16, e4m3 or e5m2 (dtype %d)",
                         int(d->dtype));
    if (!is_float(d->out))
        return fail_with(TPGEMM_ERR_DTYPE, "the output must be f16, bf16 or f32 (out %d)",
                         int(d->out));
    return check_act(d->act);
}

tpg::LinearOp linear_op(const void* A, const void* W, const tpgemm_linear_desc& d, bool gated = false) {
    tpg::LinearOp op{};
    op.M = d.M;
    op.N = d.N;
    op.K = d.K;
    op.dtype = d.dtype;
    op.a = {A, dense(d.lda, d.K), 0};
    op.b = {W, dense(d.ldw, d.K), 0};
    op.e.act = d.act;
    op.e.out = d.out;
    op.gated = gated;
    return op;
}

// Whether the tokens' rows are worth a copy to rows that start on 128-byte
// lines. With few tokens every tile reads all of them, from L2, and a row's
// stage that takes two lines takes twice as long there; with large weights that
// is more than the 2 us of a copy (f16, lines of 16 bytes off, without / with:
// 96 x 16384 x 4096 32.5 / 27.5 us, 144 x 8192 x 8192 39.7 / 29.5; without
// gain at 96 x 4096 x 4096, 12.2, and 32 x 16384 x 4096, 25.8).
bool tokens_on_lines(const tpg::LinearOp& op) {
    return op.M >= 48 && op.M <= 256 && weight_rows(op) * op.K * elem_size(op.dtype) >= int64_t(64) << 20;
}

struct LinearLayout {
    size_t total = 0;
    Aligned a, w;
};

LinearLayout linear_layout(const tpg::LinearOp& op) {
    LinearLayout L;
    if (takes_few(op)) return L;
    L.a = plan_aligned(op.a, op.M, op.K, op.dtype, &L.total, tokens_on_lines(op));
    L.w = plan_aligned(op.b, weight_rows(op), op.K, op.dtype, &L.total);
    return L;
}

// ----------------------------------------------------- linear layer, backward
struct GradLayout {
    size_t dz = 0, partial = 0, total = 0;
    size_t rest = 0, rest_scale = 0;  // of dZ, for a 32-bit dW of the gated layer
    int64_t lddz = 0;
    Aligned dy, a, w;  // copies (dY's only where it is dZ itself)
};

GradLayout grad_layout(const void* dY, const void* A, const void* W,
                       const tpgemm_linear_grad_desc& d, bool gated = false) {
    GradLayout L;
    if (d.M == 0 || d.N == 0) return L;
    const int64_t rows = gated ? 2 * d.N : d.N;
    if (gated || d.act != TPGEMM_ACT_NONE) {
        L.lddz = int64_t(align_up(size_t(rows), 64));  // whole 128-byte lines
        L.dz = L.total;
        L.total = align_up(L.total + size_t(d.M) * size_t(L.lddz) * 2, 256);
        if (gated && d.grad == TPGEMM_ELEM_F32) {
            L.rest = L.total;
            L.rest_scale = align_up(L.rest + size_t(d.M) * size_t(L.lddz) * 2, 256);
            L.total = align_up(L.rest_scale + size_t(rows) * 4, 256);
        }
    } else if (d.K > 0) {
        L.dy = plan_aligned({dY, dense(d.lddy, d.N), 0}, d.M, d.N, d.dtype, &L.total);
    }
    const int strips = gated ? tpg::gated_grad_strips(d.M, d.N) : tpg::act_grad_strips(d.M, d.N);
    L.partial = L.total;
    if (strips > 1) L.total = align_up(L.total + size_t(strips) * size_t(rows) * 4, 256);
    if (d.K > 0) {
        L.a = plan_aligned({A, dense(d.lda, d.K), 0}, d.M, d.K, d.dtype, &L.total);
        L.w = plan_aligned({W, dense(d.ldw, d.K), 0}, rows, d.K, d.dtype, &L.total);
    }
    return L;
}

tpgemm_status check_linear_grad_desc(const tpgemm_linear_grad_desc* d, bool gated = false) {
    if (!d) return fail_with(TPGEMM_ERR_NULL, "the description is NULL");
    TPG_TRY(check_dim("M", d->M, 0));
    TPG_TRY(check_dim("N", d->N, 0));
    TPG_TRY(check_dim("K", d->K, 0));
    if (gated) TPG_TRY(check_dim("2 N", 2 * d->N, 0));
    if (!is_16bit(d->dtype))
        return fail_with(TPGEMM_ERR_DTYPE, "the operands must be f16 or bf16 (dtype %d)",
                         int(d->dtype));
    if (!is_float(d->grad))
        return fail_with(TPGEMM_ERR_DTYPE, "the gradients must be f16, bf16 or f32 (grad %d)",
                         int(d->grad));
    return check_act(d->act);
}

// The linear layer and, gated, its form with two halves of weights (see LinearOp).
tpgemm_status linear_forward(bool gated, void* Y, void* Z, const void* A, const void* W, const float* scale_a,
                             const float* scale_w, const void* bias, const void* R, const tpgemm_linear_desc* d,
                             void* workspace, size_t workspace_bytes, void* stream) {
    TPG_TRY(check_linear_desc(d, gated));
    const int64_t M = d->M, N = d->N, K = d->K, rows = gated ? 2 * N : N;
    if ((scale_a || scale_w) && !is_fp8(d->dtype))
        return fail_with(TPGEMM_ERR_DTYPE, "scale_a and scale_w need e4m3 or e5m2 operands");
    Mat out[2] = {{"Y", Y, M, N, dense(d->ldy, N), d->out}, {"Z", Z, M, rows, dense(d->ldz, rows), d->out}};
    Mat in[6] = {{"A", A, M, K, dense(d->lda, K), d->dtype},
                 {"W", W, rows, K, dense(d->ldw, K), d->dtype},
                 {"R", R, M, N, dense(d->ldr, N), d->out},
                 vec("bias", bias, rows, d->out),
                 vec("scale_a", scale_a, M, TPGEMM_ELEM_F32),
                 vec("scale_w", scale_w, rows, TPGEMM_ELEM_F32)};
    if (M == 0 || N == 0) return TPGEMM_OK;
    TPG_TRY(check_mat(out[0], true));
    TPG_TRY(check_mat(out[1], false));
    for (int i = 0; i < 6; ++i) TPG_TRY(check_mat(in[i], i < 2));
    const Pair y_is_r[1] = {{0, 2}};
    TPG_TRY(check_overlap(out, 2, in, 6, y_is_r, 1));
    tpg::LinearOp op = linear_op(A, W, *d, gated);
    op.e = {Y, Z, R, bias, scale_a, scale_w, out[0].ld, out[1].ld, in[2].ld, d->act, d->out};
    const LinearLayout L = linear_layout(op);
    const size_t need = L.total;
    const Mat all[8] = {out[0], out[1], in[0], in[1], in[2], in[3], in[4], in[5]};
    TPG_TRY(check_workspace(workspace, workspace_bytes, need, all, 8));
    int sms = 0;
    TPG_TRY(tpg::require_device(&sms));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    tpg::AlignJobs copies{};
    use_aligned(L.a, &op.a, M, K, d->dtype, ws, &copies);
    use_aligned(L.w, &op.b, rows, K, d->dtype, ws, &copies);
    TPG_TRY(launched(tpg::launch_align_rows(copies, st), "operand copy launch"));
    return run_product(op, sms, st);
}

// Gradients of both.
tpgemm_status linear_gradients(bool gated, void* dA, void* dW, void* dbias, const void* dY, const void* A,
                               const void* W, const void* Z, const tpgemm_linear_grad_desc* d, void* workspace,
                               size_t workspace_bytes, void* stream) {
    TPG_TRY(check_linear_grad_desc(d, gated));
    // (Of the gated layer dZ has 2 N columns: `rows` of W.)
    const int64_t M = d->M, N = d->N, K = d->K, rows = gated ? 2 * N : N;
    const bool act = gated || d->act != TPGEMM_ACT_NONE;
    Mat out[3] = {{"dA", dA, M, K, dense(d->ldda, K), d->dtype},
                  {"dW", dW, rows, K, dense(d->lddw, K), d->grad},
                  vec("dbias", dbias, rows, d->grad)};
    Mat in[4] = {{"dY", dY, M, N, dense(d->lddy, N), d->dtype},
                 {"A", A, M, K, dense(d->lda, K), d->dtype},
                 {"W", W, rows, K, dense(d->ldw, K), d->dtype},
                 {"Z", act ? Z : nullptr, M, rows, dense(d->ldz, rows), d->dtype}};
    for (int i = 0; i < 3; ++i) TPG_TRY(check_mat(out[i], false));
    TPG_TRY(check_mat(in[0], dA || dW || dbias));
    TPG_TRY(check_mat(in[1], dW != nullptr));
    TPG_TRY(check_mat(in[2], dA != nullptr));
    TPG_TRY(check_mat(in[3], act));
    TPG_TRY(check_overlap(out, 3, in, 4, nullptr, 0));
    const GradLayout L = grad_layout(dY, A, W, *d, gated);
    const Mat all[7] = {out[0], out[1], out[2], in[0], in[1], in[2], in[3]};
    if (dA || dW || dbias)
        TPG_TRY(check_workspace(workspace, workspace_bytes, L.total, all, 7));
    int sms = 0;
    TPG_TRY(tpg::require_device(&sms));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    const size_t gs = size_t(elem_size(d->grad));
    // Sums over nothing are zero.
    if (M == 0) {
        if (dW && N > 0 && K > 0)
            TPG_TRY(launched(cudaMemset2DAsync(dW, size_t(out[1].ld) * gs, 0, size_t(K) * gs,
                                               size_t(rows), st), "zero dW"));
        if (dbias && N > 0)
            TPG_TRY(launched(cudaMemsetAsync(dbias, 0, size_t(rows) * gs, st), "zero dbias"));
        return TPGEMM_OK;
    }
    if (N == 0) {
        if (dA && K > 0)
            TPG_TRY(launched(cudaMemset2DAsync(dA, size_t(out[0].ld) * 2, 0, size_t(K) * 2,
                                               size_t(M), st), "zero dA"));
        return TPGEMM_OK;
    }
    const void* dz = dY;
    int64_t lddz = in[0].ld;
    if (dbias || (act && (dA || dW))) {
        tpg::ActGradOp g{M, N, dY, in[3].p, in[0].ld, in[3].ld,
                         (act && (dA || dW)) ? ws + L.dz : nullptr, L.lddz,
                         reinterpret_cast<float*>(ws + L.partial), dbias,
                         d->dtype, d->act, d->grad};
        tpg::DzRest rest{};
        if (L.rest && dW) rest = {ws + L.rest, reinterpret_cast<float*>(ws + L.rest_scale)};
        TPG_TRY(launched(gated ? tpg::launch_gated_grad(g, rest, st) : tpg::launch_act_grad(g, st),
                         "activation gradient launch"));
    }
    if (act) {
        dz = ws + L.dz;
        lddz = L.lddz;
    }
    if (K == 0) return TPGEMM_OK;
    if (!dA && !dW) return TPGEMM_OK;
    tpg::Operand oz{dz, lddz, 0}, oa{A, in[1].ld, 0}, ow{W, in[2].ld, 0};
    tpg::AlignJobs copies{};
    use_aligned(L.dy, &oz, M, rows, d->dtype, ws, &copies);
    if (dA) use_aligned(L.w, &ow, rows, K, d->dtype, ws, &copies);
    if (dW) use_aligned(L.a, &oa, M, K, d->dtype, ws, &copies);
    TPG_TRY(launched(tpg::launch_align_rows(copies, st), "operand copy launch"));
    if (dA) {  // [M, K] = dZ [M, rows] . W: the reduction runs along W's rows
        tpg::LinearOp op{M, K, rows, d->dtype, oz, {ow.p, ow.ld, 1},
                         {dA, nullptr, nullptr, nullptr, nullptr, nullptr, out[0].ld, 0, 0,
                          TPGEMM_ACT_NONE, d->dtype}};
        TPG_TRY(run_product(op, sms, st));
    }
    if (dW) {  // [rows, K] = dZ^T . A: along the rows of both
        tpg::LinearOp op{rows, K, M, d->dtype, {oz.p, oz.ld, 1}, {oa.p, oa.ld, 1},
                         {dW, nullptr, nullptr, nullptr, nullptr, nullptr, out[1].ld, 0, 0,
                          TPGEMM_ACT_NONE, d->grad}};
        // (A 32-bit dW of the gated layer: some tokens after the others, dW += ..., and
        // then scale rest^T . A.)
        const int64_t parts = L.rest ? (M + tpg::kLongSum - 1) / tpg::kLongSum : 1;
        for (int64_t i = 0; i < parts; ++i) {
            const int64_t begin = M * i / parts / 64 * 64, end = i + 1 == parts ? M : M * (i + 1) / parts / 64 * 64;
            op.K = end - begin;
            op.a.p = static_cast<const uint8_t*>(oz.p) + begin * oz.ld * 2;
            op.b.p = static_cast<const uint8_t*>(oa.p) + begin * oa.ld * 2;
            op.e.R = i > 0 ? dW : nullptr;
            op.e.ldr = out[1].ld;
            TPG_TRY(run_product(op, sms, st));
        }
        if (L.rest) {
            op.K = M;
            op.a.p = ws + L.rest;
            op.b.p = oa.p;
            op.e.R = dW;
            op.e.rest = 1;
            op.e.sa = reinterpret_cast<const float*>(ws + L.rest_scale);
            TPG_TRY(run_product(op, sms, st));
        }
    }
    return TPGEMM_OK;
}

// Dropout's numbers; `in` gets the counter's place, for the overlap check.
tpgemm_status check_drop(const tpgemm_drop& d, tpg::Drop* drop, Mat* in) {
    *in = {"counter", nullptr, 1, 8, 8, TPGEMM_ELEM_E4M3};
    *drop = {};
    if (!(d.p >= 0.0 && d.p < 1.0))
        return fail_with(TPGEMM_ERR_SHAPE, "p=%g must be at least 0 and below 1", d.p);
    if (d.p == 0.0) return TPGEMM_OK;
    if (reinterpret_cast<uintptr_t>(d.counter) % 8)
        return fail_with(TPGEMM_ERR_ALIGN, "counter=%p is not 8-byte aligned",
                         static_cast<const void*>(d.counter));
    in->p = d.counter;
    const double t = std::nearbyint(d.p * 4294967296.0);
    tpg::drop_keys(drop, d.seed);
    drop->offset = d.offset;
    drop->counter = d.counter;
    drop->threshold = t < 4294967295.0 ? uint32_t(t) : 0xffffffffu;
    drop->scale = float(1.0 / (1.0 - d.p));
    drop->on = 1;
    return TPGEMM_OK;
}

size_t layernorm_grad_ws(int64_t rows, int64_t cols) {
    return align_up(size_t(tpg::layernorm_grad_strips(rows, cols)) * size_t(cols) * 8, 256);
}

size_t rmsnorm_grad_ws(int64_t rows, int64_t cols) {
    return align_up(size_t(tpg::rmsnorm_grad_strips(rows, cols)) * size_t(cols) * 4, 256);
}

}  // namespace

extern "C" {

size_t tpgemm_linear_workspace_bytes(const void* A, const void* W, const tpgemm_linear_desc* d) {
    tpg::set_error_detail("");
    if (check_linear_desc(d) != TPGEMM_OK || d->M == 0 || d->N == 0) return 0;
    return linear_layout(linear_op(A, W, *d)).total;
}

tpgemm_status tpgemm_linear(void* Y, void* Z, const void* A, const void* W, const float* scale_a,
                            const float* scale_w, const void* bias, const void* R,
                            const tpgemm_linear_desc* d, void* workspace, size_t workspace_bytes,
                            void* stream) {
    tpg::set_error_detail("");
    return linear_forward(false, Y, Z, A, W, scale_a, scale_w, bias, R, d, workspace, workspace_bytes, stream);
}

size_t tpgemm_linear_backward_workspace_bytes(const void* dY, const void* A, const void* W,
                                              const tpgemm_linear_grad_desc* d) {
    tpg::set_error_detail("");
    if (check_linear_grad_desc(d) != TPGEMM_OK) return 0;
    return grad_layout(dY, A, W, *d).total;
}

tpgemm_status tpgemm_linear_backward(void* dA, void* dW, void* dbias, const void* dY,
                                     const void* A, const void* W, const void* Z,
                                     const tpgemm_linear_grad_desc* d, void* workspace,
                                     size_t workspace_bytes, void* stream) {
    tpg::set_error_detail("");
    return linear_gradients(false, dA, dW, dbias, dY, A, W, Z, d, workspace, workspace_bytes, stream);
}

size_t tpgemm_gated_linear_workspace_bytes(const void* A, const void* W, const tpgemm_linear_desc* d) {
    tpg::set_error_detail("");
    if (check_linear_desc(d, true) != TPGEMM_OK || d->M == 0 || d->N == 0) return 0;
    return linear_layout(linear_op(A, W, *d, true)).total;
}

tpgemm_status tpgemm_gated_linear(void* Y, void* Z, const void* A, const void* W, const float* scale_a,
                                  const float* scale_w, const void* bias, const tpgemm_linear_desc* d,
                                  void* workspace, size_t workspace_bytes, void* stream) {
    tpg::set_error_detail("");
    return linear_forward(true, Y, Z, A, W, scale_a, scale_w, bias, nullptr, d, workspace, workspace_bytes, stream);
}

size_t tpgemm_gated_linear_backward_workspace_bytes(const void* dY, const void* A, const void* W,
                                                    const tpgemm_linear_grad_desc* d) {
    tpg::set_error_detail("");
    if (check_linear_grad_desc(d, true) != TPGEMM_OK) return 0;
    return grad_layout(dY, A, W, *d, true).total;
}

tpgemm_status tpgemm_gated_linear_backward(void* dA, void* dW, void* dbias, const void* dY, const void* A,
                                           const void* W, const void* Z, const tpgemm_linear_grad_desc* d,
                                           void* workspace, size_t workspace_bytes, void* stream) {
    tpg::set_error_detail("");
    return linear_gradients(true, dA, dW, dbias, dY, A, W, Z, d, workspace, workspace_bytes, stream);
}

tpgemm_status tpgemm_rmsnorm(void* Y, void* H, void* scale, float* rstd, const void* X,
                             const void* R, const void* gamma, const tpgemm_rmsnorm_desc* d,
                             void* stream) {
    tpg::set_error_detail("");
    if (!d) return fail_with(TPGEMM_ERR_NULL, "the description is NULL");
    TPG_TRY(check_dim("rows", d->rows, 0));
    TPG_TRY(check_dim("cols", d->cols, 1));
    if (!is_float(d->x)) return fail_with(TPGEMM_ERR_DTYPE, "X must be f16, bf16 or f32 (%d)", int(d->x));
    if (d->gamma != d->x && d->gamma != TPGEMM_ELEM_F32)
        return fail_with(TPGEMM_ERR_DTYPE, "gamma must be of X's type or f32 (%d)", int(d->gamma));
    if (d->scale != TPGEMM_SCALE_NONE && d->scale != TPGEMM_SCALE_ROW && d->scale != TPGEMM_SCALE_MX)
        return fail_with(TPGEMM_ERR_DTYPE, "scale mode %d is not one of tpgemm_scale_mode", int(d->scale));
    if (d->scale == TPGEMM_SCALE_NONE ? !is_float(d->y) : !is_fp8(d->y))
        return fail_with(TPGEMM_ERR_DTYPE,
                         "Y must be f16, bf16 or f32 without scales and e4m3 or e5m2 with them (%d)",
                         int(d->y));
    if (!(d->eps >= 0.f))
        return fail_with(TPGEMM_ERR_SHAPE, "eps=%g must not be negative", double(d->eps));
    const int64_t rows = d->rows, cols = d->cols;
    if (rows == 0) return TPGEMM_OK;
    const bool row = d->scale == TPGEMM_SCALE_ROW, mx = d->scale == TPGEMM_SCALE_MX;
    const int64_t blocks = (cols + 31) / 32;
    Mat out[4] = {{"Y", Y, rows, cols, dense(d->ldy, cols), d->y},
                  {"H", H, rows, cols, dense(d->ldh, cols), d->x},
                  {"scale", (row || mx) ? scale : nullptr, 1, row ? rows : rows * blocks,
                   row ? rows : rows * blocks, row ? TPGEMM_ELEM_F32 : TPGEMM_ELEM_E4M3},
                  vec("rstd", rstd, rows, TPGEMM_ELEM_F32)};
    Mat in[3] = {{"X", X, rows, cols, dense(d->ldx, cols), d->x},
                 {"R", R, rows, cols, dense(d->ldr, cols), d->x},
                 vec("gamma", gamma, cols, d->gamma)};
    TPG_TRY(check_mat(out[0], true));
    TPG_TRY(check_mat(out[1], false));
    TPG_TRY(check_mat(out[2], row || mx));
    TPG_TRY(check_mat(out[3], false));
    TPG_TRY(check_mat(in[0], true));
    TPG_TRY(check_mat(in[1], false));
    TPG_TRY(check_mat(in[2], true));
    const Pair pairs[4] = {{1, 0}, {1, 1}, {0, 0}, {0, 1}};
    TPG_TRY(check_overlap(out, 4, in, 3, pairs, H ? 2 : 4));
    int sms = 0;
    TPG_TRY(tpg::require_device(&sms));
    tpg::RmsNormOp op{rows, cols, X, R, gamma, H, Y, scale, rstd, in[0].ld, in[1].ld, out[1].ld,
                      out[0].ld, d->x, d->gamma, d->y, d->scale, d->eps};
    return launched(tpg::launch_rmsnorm(op, static_cast<cudaStream_t>(stream)), "norm launch");
}

size_t tpgemm_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t cols) {
    if (rows <= 0 || cols <= 0 || rows >= kMaxDim || cols >= kMaxDim) return 0;
    return rmsnorm_grad_ws(rows, cols);
}

tpgemm_status tpgemm_rmsnorm_backward(void* dX, void* dgamma, const void* dY, const void* H,
                                      const float* rstd, const void* gamma, const void* dH,
                                      const tpgemm_rmsnorm_grad_desc* d, void* workspace,
                                      size_t workspace_bytes, void* stream) {
    tpg::set_error_detail("");
    if (!d) return fail_with(TPGEMM_ERR_NULL, "the description is NULL");
    TPG_TRY(check_dim("rows", d->rows, 0));
    TPG_TRY(check_dim("cols", d->cols, 1));
    if (!is_float(d->x)) return fail_with(TPGEMM_ERR_DTYPE, "dY must be f16, bf16 or f32 (%d)", int(d->x));
    if (d->gamma != d->x && d->gamma != TPGEMM_ELEM_F32)
        return fail_with(TPGEMM_ERR_DTYPE, "gamma must be of dY's type or f32 (%d)", int(d->gamma));
    if (!is_float(d->grad))
        return fail_with(TPGEMM_ERR_DTYPE, "dgamma must be f16, bf16 or f32 (%d)", int(d->grad));
    const int64_t rows = d->rows, cols = d->cols;
    const bool any = dX || dgamma;
    Mat out[2] = {{"dX", dX, rows, cols, dense(d->lddx, cols), d->x},
                  vec("dgamma", dgamma, cols, d->grad)};
    Mat in[5] = {{"dY", dY, rows, cols, dense(d->lddy, cols), d->x},
                 {"H", H, rows, cols, dense(d->ldh, cols), d->x},
                 {"dH", dH, rows, cols, dense(d->lddh, cols), d->x},
                 vec("rstd", rstd, rows, TPGEMM_ELEM_F32),
                 vec("gamma", gamma, cols, d->gamma)};
    for (Mat& m : out) TPG_TRY(check_mat(m, false));
    for (int i = 0; i < 5; ++i) TPG_TRY(check_mat(in[i], any && rows > 0 && i != 2 && (i != 4 || dX)));
    const Pair pairs[3] = {{0, 0}, {0, 1}, {0, 2}};
    TPG_TRY(check_overlap(out, 2, in, 5, pairs, 3));
    const Mat all[7] = {out[0], out[1], in[0], in[1], in[2], in[3], in[4]};
    if (dgamma && rows > 0)
        TPG_TRY(check_workspace(workspace, workspace_bytes, rmsnorm_grad_ws(rows, cols), all, 7));
    int sms = 0;
    TPG_TRY(tpg::require_device(&sms));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (rows == 0) {
        if (dgamma)
            return launched(cudaMemsetAsync(dgamma, 0, size_t(cols) * size_t(elem_size(d->grad)), st),
                            "zero dgamma");
        return TPGEMM_OK;
    }
    if (!any) return TPGEMM_OK;
    tpg::RmsNormGradOp op{rows, cols, dY, H, rstd, gamma, dH, dX, dgamma,
                          static_cast<float*>(workspace), in[0].ld, in[1].ld, in[2].ld, out[0].ld,
                          d->x, d->gamma, d->grad};
    return launched(tpg::launch_rmsnorm_grad(op, st), "norm gradient launch");
}

tpgemm_status tpgemm_dropout(void* Y, const void* X, const void* R, const tpgemm_dropout_desc* d,
                             void* stream) {
    tpg::set_error_detail("");
    if (!d) return fail_with(TPGEMM_ERR_NULL, "the description is NULL");
    TPG_TRY(check_dim("rows", d->rows, 0));
    TPG_TRY(check_dim("cols", d->cols, 0));
    if (!is_float(d->x)) return fail_with(TPGEMM_ERR_DTYPE, "X must be f16, bf16 or f32 (%d)", int(d->x));
    tpg::Drop drop;
    Mat counter;
    TPG_TRY(check_drop(d->drop, &drop, &counter));
    const int64_t rows = d->rows, cols = d->cols;
    if (rows == 0 || cols == 0) return TPGEMM_OK;
    Mat out[1] = {{"Y", Y, rows, cols, dense(d->ldy, cols), d->x}};
    Mat in[3] = {{"X", X, rows, cols, dense(d->ldx, cols), d->x},
                 {"R", R, rows, cols, dense(d->ldr, cols), d->x},
                 counter};
    TPG_TRY(check_mat(out[0], true));
    TPG_TRY(check_mat(in[0], true));
    TPG_TRY(check_mat(in[1], false));
    const Pair pairs[2] = {{0, 0}, {0, 1}};
    TPG_TRY(check_overlap(out, 1, in, 3, pairs, 2));
    int sms = 0;
    TPG_TRY(tpg::require_device(&sms));
    const tpg::DropoutOp op{rows, cols, X, R, Y, in[0].ld, in[1].ld, out[0].ld, d->x, drop};
    return launched(tpg::launch_dropout(op, static_cast<cudaStream_t>(stream)), "dropout launch");
}

tpgemm_status tpgemm_layernorm(void* Y, void* H, float* scale, float* mean, float* rstd,
                               const void* X, const void* R, const void* gamma, const void* beta,
                               const tpgemm_layernorm_desc* d, void* stream) {
    tpg::set_error_detail("");
    if (!d) return fail_with(TPGEMM_ERR_NULL, "the description is NULL");
    TPG_TRY(check_dim("rows", d->rows, 0));
    TPG_TRY(check_dim("cols", d->cols, 1));
    if (!is_float(d->x)) return fail_with(TPGEMM_ERR_DTYPE, "X must be f16, bf16 or f32 (%d)", int(d->x));
    if (d->gamma != d->x && d->gamma != TPGEMM_ELEM_F32)
        return fail_with(TPGEMM_ERR_DTYPE, "gamma and beta must be of X's type or f32 (%d)", int(d->gamma));
    if (d->scale != TPGEMM_SCALE_NONE && d->scale != TPGEMM_SCALE_ROW)
        return fail_with(TPGEMM_ERR_DTYPE, "scale mode %d must be none or row", int(d->scale));
    const bool row = d->scale == TPGEMM_SCALE_ROW;
    if (row ? !is_fp8(d->y) : !is_float(d->y))
        return fail_with(TPGEMM_ERR_DTYPE,
                         "Y must be f16, bf16 or f32 without scales and e4m3 or e5m2 with them (%d)",
                         int(d->y));
    if (!(d->eps >= 0.f))
        return fail_with(TPGEMM_ERR_SHAPE, "eps=%g must not be negative", double(d->eps));
    tpg::Drop drop;
    Mat counter;
    TPG_TRY(check_drop(d->drop, &drop, &counter));
    const int64_t rows = d->rows, cols = d->cols;
    if (rows == 0) return TPGEMM_OK;
    Mat out[5] = {{"Y", Y, rows, cols, dense(d->ldy, cols), d->y},
                  {"H", H, rows, cols, dense(d->ldh, cols), d->x},
                  vec("scale", row ? scale : nullptr, rows, TPGEMM_ELEM_F32),
                  vec("mean", mean, rows, TPGEMM_ELEM_F32),
                  vec("rstd", rstd, rows, TPGEMM_ELEM_F32)};
    Mat in[5] = {{"X", X, rows, cols, dense(d->ldx, cols), d->x},
                 {"R", R, rows, cols, dense(d->ldr, cols), d->x},
                 vec("gamma", gamma, cols, d->gamma),
                 vec("beta", beta, cols, d->gamma),
                 counter};
    for (int i = 0; i < 5; ++i) TPG_TRY(check_mat(out[i], i == 0 || (i == 2 && row)));
    for (int i = 0; i < 5; ++i) TPG_TRY(check_mat(in[i], i == 0 || i == 2));
    const Pair pairs[4] = {{1, 0}, {1, 1}, {0, 0}, {0, 1}};
    TPG_TRY(check_overlap(out, 5, in, 5, pairs, H ? 2 : 4));
    int sms = 0;
    TPG_TRY(tpg::require_device(&sms));
    const tpg::LayerNormOp op{rows, cols, X, R, gamma, beta, H, Y, scale, mean, rstd, in[0].ld, in[1].ld,
                              out[1].ld, out[0].ld, d->x, d->gamma, d->y, d->scale, d->eps, drop};
    return launched(tpg::launch_layernorm(op, static_cast<cudaStream_t>(stream)), "layer norm launch");
}

size_t tpgemm_layernorm_backward_workspace_bytes(int64_t rows, int64_t cols) {
    if (rows <= 0 || cols <= 0 || rows >= kMaxDim || cols >= kMaxDim) return 0;
    return layernorm_grad_ws(rows, cols);
}

tpgemm_status tpgemm_layernorm_backward(void* dX, void* dR, void* dgamma, void* dbeta,
                                        const void* dY, const void* H, const float* mean,
                                        const float* rstd, const void* gamma, const void* dH,
                                        const tpgemm_layernorm_grad_desc* d, void* workspace,
                                        size_t workspace_bytes, void* stream) {
    tpg::set_error_detail("");
    if (!d) return fail_with(TPGEMM_ERR_NULL, "the description is NULL");
    TPG_TRY(check_dim("rows", d->rows, 0));
    TPG_TRY(check_dim("cols", d->cols, 1));
    if (!is_float(d->x)) return fail_with(TPGEMM_ERR_DTYPE, "dY must be f16, bf16 or f32 (%d)", int(d->x));
    if (d->gamma != d->x && d->gamma != TPGEMM_ELEM_F32)
        return fail_with(TPGEMM_ERR_DTYPE, "gamma must be of dY's type or f32 (%d)", int(d->gamma));
    if (!is_float(d->grad))
        return fail_with(TPGEMM_ERR_DTYPE, "dgamma and dbeta must be f16, bf16 or f32 (%d)", int(d->grad));
    tpg::Drop drop;
    Mat counter;
    TPG_TRY(check_drop(d->drop, &drop, &counter));
    const int64_t rows = d->rows, cols = d->cols;
    const bool by_row = dX || dR, by_col = dgamma || dbeta;
    Mat out[4] = {{"dX", dX, rows, cols, dense(d->lddx, cols), d->x},
                  {"dR", dR, rows, cols, dense(d->lddr, cols), d->x},
                  vec("dgamma", dgamma, cols, d->grad),
                  vec("dbeta", dbeta, cols, d->grad)};
    Mat in[7] = {{"dY", dY, rows, cols, dense(d->lddy, cols), d->x},
                 {"H", H, rows, cols, dense(d->ldh, cols), d->x},
                 {"dH", dH, rows, cols, dense(d->lddh, cols), d->x},
                 vec("mean", mean, rows, TPGEMM_ELEM_F32),
                 vec("rstd", rstd, rows, TPGEMM_ELEM_F32),
                 vec("gamma", gamma, cols, d->gamma),
                 counter};
    for (Mat& m : out) TPG_TRY(check_mat(m, false));
    for (int i = 0; i < 7; ++i)
        TPG_TRY(check_mat(in[i], (by_row || by_col) && rows > 0 && i != 2 && i != 6 && (i != 5 || by_row)));
    const Pair pairs[6] = {{0, 0}, {0, 1}, {0, 2}, {1, 0}, {1, 1}, {1, 2}};
    TPG_TRY(check_overlap(out, 4, in, 7, pairs, 6));
    const Mat all[11] = {out[0], out[1], out[2], out[3], in[0], in[1], in[2], in[3], in[4], in[5], in[6]};
    if (by_col && rows > 0)
        TPG_TRY(check_workspace(workspace, workspace_bytes, layernorm_grad_ws(rows, cols), all, 11));
    int sms = 0;
    TPG_TRY(tpg::require_device(&sms));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (rows == 0) {
        const size_t bytes = size_t(cols) * size_t(elem_size(d->grad));
        if (dgamma) TPG_TRY(launched(cudaMemsetAsync(dgamma, 0, bytes, st), "zero dgamma"));
        if (dbeta) TPG_TRY(launched(cudaMemsetAsync(dbeta, 0, bytes, st), "zero dbeta"));
        return TPGEMM_OK;
    }
    if (!by_row && !by_col) return TPGEMM_OK;
    const tpg::LayerNormGradOp op{rows, cols, dY, H, mean, rstd, gamma, dH, dX, dR, dgamma, dbeta,
                                  by_col ? static_cast<float*>(workspace) : nullptr, in[0].ld, in[1].ld,
                                  in[2].ld, out[0].ld, out[1].ld, d->x, d->gamma, d->grad, drop};
    return launched(tpg::launch_layernorm_grad(op, st), "layer norm gradient launch");
}

}  // extern "C"
