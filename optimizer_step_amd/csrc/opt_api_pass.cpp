// opt_api_pass.cpp -- the C ABI of the training-pass operators: argument
// checks and launches.  Nothing here holds state: what an operator needs
// besides its tensors the caller passes.
#include <hip/hip_runtime.h>

#include <cmath>
#include <initializer_list>

#include "opt_pass.h"
#include "opt_step.h"

namespace optstep {

int report(int code, const char *fmt, ...);
int report_hip(hipError_t e, const char *what);

hipError_t launch_dropout(int dt, const DropArgs &a, hipStream_t st);
hipError_t launch_rms_norm(int dt, const NormArgs &a, hipStream_t st);
hipError_t launch_rms_norm_grad(int dt, const NormGradArgs &a, float *dw, int accumulate, hipStream_t st);
hipError_t launch_block_cast(int dt, const CastArgs &a, int square, hipStream_t st);
hipError_t launch_block_matmul(int dt, const MatmulArgs &a, hipStream_t st);
hipError_t launch_gated_act(int dt, int act, const GateArgs &a, hipStream_t st);
hipError_t launch_gated_act_grad(int dt, int act, const GateGradArgs &a, hipStream_t st);
hipError_t launch_block_restore(int dt, const RestoreArgs &a, hipStream_t st);
hipError_t launch_head_norm(int dt, const HeadArgs &a, hipStream_t st);
hipError_t launch_head_norm_grad(int dt, int coded, const HeadGradArgs &a, float *dwq, float *dwk, int accumulate, hipStream_t st);

namespace {

constexpr int64_t kMaxElems = (int64_t)1 << 46;
constexpr int64_t kMaxIndex = (int64_t)1 << 60;
constexpr int64_t kMaxSide = (int64_t)1 << 31;

bool at(const void *p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
int64_t up(int64_t n, int64_t m) { return (n + m - 1) / m * m; }
size_t size_of(int32_t dt) { return dt == OPT_F32 ? 4 : 2; }

int check_dtype(int32_t dt, const char *what)
{
    if (dt != OPT_F32 && dt != OPT_BF16 && dt != OPT_F16) return report(OPT_EINVAL, "unknown %s %d", what, dt);
    return OPT_OK;
}

int check_sides(int64_t rows, int64_t cols)
{
    if (rows < 0 || cols < 0) return report(OPT_EINVAL, "negative size");
    if (rows >= kMaxSide || cols >= kMaxSide) return report(OPT_EINVAL, "rows and columns must be below 2^31");
    return OPT_OK;
}

// Rows of ld elements of which cols are used (rows, cols > 0).
int check_ld(const char *what, int64_t ld, int64_t rows, int64_t cols)
{
    if (rows == 1) return cols <= kMaxElems ? OPT_OK : report(OPT_EINVAL, "%s is too long", what);
    if (ld < cols) return report(OPT_EINVAL, "%s: leading dimension %lld below its %lld columns", what, (long long)ld, (long long)cols);
    if (ld > kMaxElems / rows) return report(OPT_EINVAL, "%s: rows times leading dimension above 2^46", what);
    return OPT_OK;
}

int check_matrix(const char *what, const void *p, int64_t ld, int64_t rows, int64_t cols, size_t size)
{
    if (!p) return report(OPT_EINVAL, "%s is NULL", what);
    if (!at(p, size)) return report(OPT_EALIGN, "%s must be aligned to its %d-byte elements", what, (int)size);
    return check_ld(what, ld, rows, cols);
}

// A block-coded matrix of `rows` rows of `bytes` used code bytes.
int check_codes(const char *what, const opt_codes &q, int64_t rows, int64_t bytes)
{
    int rc;
    if (!q.codes || !q.scales) return report(OPT_EINVAL, "%s: codes or scales is NULL", what);
    if (!at(q.codes, 16) || (rows > 1 && q.ld % 16 != 0))
        return report(OPT_EALIGN, "%s: codes must be 16-byte aligned, rows of a multiple of 16 bytes", what);
    if (!at(q.scales, 4) || q.lds % 4 != 0)
        return report(OPT_EALIGN, "%s: scales must be 4-byte aligned, a multiple of 4 bytes apart", what);
    if ((rc = check_ld(what, q.ld, rows, up(bytes, 16))) != OPT_OK) return rc;
    if (q.lds < rows) return report(OPT_EINVAL, "%s: %lld scales a block row for %lld rows", what, (long long)q.lds, (long long)rows);
    if (q.lds > kMaxElems / (up(bytes, kCodeBlock) / kCodeBlock)) return report(OPT_EINVAL, "%s: too many scales", what);
    return OPT_OK;
}

Codes codes_of(const opt_codes &q) { return Codes{q.codes, q.ld, q.scales, q.lds}; }

// An optional output.
int check_more(const char *what, const void *p, int64_t ld, int64_t rows, int64_t cols, size_t size)
{
    return p ? check_matrix(what, p, ld, rows, cols, size) : OPT_OK;
}

int check_more(const char *what, const opt_codes &q, int64_t rows, int64_t bytes)
{
    return q.codes ? check_codes(what, q, rows, bytes) : OPT_OK;
}

// Coded outputs of one call: each in buffers of its own.
int check_apart(std::initializer_list<const opt_codes *> out)
{
    for (const opt_codes *a : out)
        for (const opt_codes *b : out) {
            if (a == b) break;
            if (a->codes && b->codes && (a->codes == b->codes || a->scales == b->scales))
                return report(OPT_EINVAL, "two coded results have the same buffer");
        }
    return OPT_OK;
}

// A result over an input lies as the input does: elsewhere a workgroup would
// write what another still reads.
int check_over(const char *what, const void *out, int64_t ldo, const void *in, int64_t ldi, int64_t rows)
{
    if (out && out == in && rows > 1 && ldo != ldi) return report(OPT_EINVAL, "%s over an input must have its leading dimension", what);
    return OPT_OK;
}

int check_over(const char *what, const void *out, int64_t ot, int64_t oh, const void *in, int64_t it, int64_t ih, int64_t tokens, int64_t heads)
{
    if (out == in && ((tokens > 1 && ot != it) || (heads > 1 && oh != ih))) return report(OPT_EINVAL, "%s over an input must have its strides", what);
    return OPT_OK;
}

int check_act(int32_t act)
{
    return act == OPT_SILU || act == OPT_GELU ? OPT_OK : report(OPT_EINVAL, "unknown activation %d", act);
}

// Heads of dim elements, `token` and `head` elements apart.  Outputs lie apart
// from each other: heads within a token, or tokens within a head.
int check_heads(const char *what, const void *p, int64_t token, int64_t head, int64_t tokens, int64_t heads, int64_t dim, size_t size, bool out)
{
    if (!p) return report(OPT_EINVAL, "%s is NULL", what);
    if (!at(p, size)) return report(OPT_EALIGN, "%s must be aligned to its %d-byte elements", what, (int)size);
    if ((tokens > 1 && token < 0) || (heads > 1 && head < 0)) return report(OPT_EINVAL, "%s: negative stride", what);
    if ((tokens > 1 && token > kMaxElems / tokens) || (heads > 1 && head > kMaxElems / heads))
        return report(OPT_EINVAL, "%s: tokens or heads times their stride above 2^46", what);
    if (out) {
        const bool inner = heads == 1 || head >= dim, outer = tokens == 1 || token >= dim;
        const bool by_token = tokens == 1 || token >= (heads - 1) * head + dim, by_head = heads == 1 || head >= (tokens - 1) * token + dim;
        if (!inner || !outer || !(by_token || by_head)) return report(OPT_EINVAL, "%s: its heads overlap", what);
    }
    return OPT_OK;
}

int check_turn(int64_t tokens, int32_t dim, int32_t rot, int32_t dtype, int32_t w_dtype, int32_t interleaved, double eps)
{
    int rc;
    if ((rc = check_dtype(dtype, "dtype")) != OPT_OK) return rc;
    if ((rc = check_dtype(w_dtype, "w_dtype")) != OPT_OK) return rc;
    if (tokens < 0 || tokens >= kMaxSide) return report(OPT_EINVAL, "tokens must lie in [0, 2^31)");
    if (dim < 1) return report(OPT_EINVAL, "dim must be positive");
    if (dim > kMaxHeadDim) return report(OPT_EUNSUPPORTED, "heads above %d elements", kMaxHeadDim);
    if (rot < 0 || rot > dim || rot % 2 != 0) return report(OPT_EINVAL, "rot must be even, in [0, dim]");
    if (interleaved != 0 && interleaved != 1) return report(OPT_EINVAL, "interleaved must be 0 or 1");
    if (!(eps >= 0.0) || std::isinf(eps)) return report(OPT_EINVAL, "eps must be a non-negative number");
    return OPT_OK;
}

int check_table(const opt_head_table &t, int64_t tokens, int32_t rot)
{
    if (rot == 0 || tokens == 0) return OPT_OK;
    if (t.position_bits != 32 && t.position_bits != 64) return report(OPT_EINVAL, "position_bits must be 32 or 64");
    if (t.rows < 1 || t.rows >= kMaxSide) return report(OPT_EINVAL, "the table's rows must lie in [1, 2^31)");
    int rc;
    if ((rc = check_matrix("table", t.cos_sin, t.ld, t.rows, rot, 4)) != OPT_OK) return rc;
    if (!t.positions && tokens > t.rows) return report(OPT_EINVAL, "the table holds %lld positions of %lld", (long long)t.rows, (long long)tokens);
    if (!at(t.positions, (size_t)t.position_bits / 8)) return report(OPT_EALIGN, "positions must be aligned to their elements");
    return OPT_OK;
}

int check_count(const char *what, int64_t heads, int64_t tokens, bool coded)
{
    if (heads < 0 || heads >= 65536) return report(OPT_EINVAL, "%s: heads must lie in [0, 65536)", what);
    if (coded && heads * tokens >= kMaxSide) return report(OPT_EINVAL, "%s: coded tokens times heads must be below 2^31", what);
    return OPT_OK;
}

HeadTurn turn_of(int64_t tokens, int32_t dim, int32_t rot, int32_t w_dtype, int32_t interleaved, double eps, const opt_head_table &t)
{
    HeadTurn r{};
    r.tokens = tokens;
    r.table_rows = t.rows;
    r.ldt = t.ld;
    r.table = t.cos_sin;
    r.positions = t.positions;
    r.dim = dim;
    r.rot = rot;
    r.wide_positions = t.position_bits == 64;
    r.neighbours = interleaved;
    r.w_dtype = w_dtype;
    r.eps = eps;
    r.inv_dim = 1.0 / (double)dim;
    return r;
}

int done(hipError_t e, const char *what) { return e == hipSuccess ? OPT_OK : report_hip(e, what); }

}  // namespace
}  // namespace optstep

using namespace optstep;

extern "C" {

int opt_dropout(const void *x, const void *residual, void *out, int64_t n, int32_t dtype, double p, uint64_t seed,
                uint64_t offset, int64_t index_base, void *stream)
{
    int rc;
    if ((rc = check_dtype(dtype, "dtype")) != OPT_OK) return rc;
    if (n < 0 || n > kMaxElems) return report(OPT_EINVAL, "n must lie in [0, 2^46]");
    if (!(p >= 0.0 && p <= 1.0)) return report(OPT_EINVAL, "p must lie in [0, 1]");
    if (index_base < 0 || index_base % 8 != 0) return report(OPT_EINVAL, "index_base must be a non-negative multiple of 8");
    if (index_base > kMaxIndex - n) return report(OPT_EINVAL, "index_base + n above 2^60");
    if (n == 0) return OPT_OK;
    if (!x || !out) return report(OPT_EINVAL, "x or out is NULL");
    const size_t size = size_of(dtype);
    if (!at(x, size) || !at(residual, size) || !at(out, size))
        return report(OPT_EALIGN, "x, residual and out must be aligned to their elements");
    DropArgs a{};
    a.x = x;
    a.res = residual;
    a.out = out;
    a.n = n;
    a.base8 = index_base / 8;
    a.seed = seed;
    a.offset = offset;
    a.threshold = (uint32_t)floor(p * 65536.0 + 0.5);
    a.scale = a.threshold < 65536u ? (float)(1.0 / (1.0 - a.threshold / 65536.0)) : 0.0f;
    return done(launch_dropout(dtype, a, (hipStream_t)stream), "dropout launch");
}

int opt_rms_norm(const opt_norm *n, void *stream)
{
    int rc;
    if (!n) return report(OPT_EINVAL, "the argument record is NULL");
    if ((rc = check_dtype(n->dtype, "dtype")) != OPT_OK) return rc;
    if ((rc = check_dtype(n->w_dtype, "w_dtype")) != OPT_OK) return rc;
    if ((rc = check_sides(n->rows, n->cols)) != OPT_OK) return rc;
    if (!(n->eps >= 0.0) || std::isinf(n->eps)) return report(OPT_EINVAL, "eps must be a non-negative number");
    if (n->rows == 0 || n->cols == 0) return OPT_OK;
    if (n->cols > kMaxNormCols) return report(OPT_EUNSUPPORTED, "rows above %lld columns", (long long)kMaxNormCols);
    if (!n->y && !n->q.codes) return report(OPT_EINVAL, "neither y nor q is given");
    const size_t size = size_of(n->dtype);
    if ((rc = check_matrix("x", n->x, n->ldx, n->rows, n->cols, size)) != OPT_OK) return rc;
    if (n->residual && (rc = check_matrix("residual", n->residual, n->ldr, n->rows, n->cols, size)) != OPT_OK) return rc;
    if ((rc = check_matrix("weight", n->weight, n->cols, 1, n->cols, size_of(n->w_dtype))) != OPT_OK) return rc;
    if (n->h && (rc = check_matrix("h", n->h, n->ldh, n->rows, n->cols, size)) != OPT_OK) return rc;
    if (n->y && (rc = check_matrix("y", n->y, n->ldy, n->rows, n->cols, size)) != OPT_OK) return rc;
    if (n->h && n->h == n->y) return report(OPT_EINVAL, "h and y must be different matrices");
    if (n->q.codes && (rc = check_codes("q", n->q, n->rows, n->cols)) != OPT_OK) return rc;
    NormArgs a{};
    a.rows = n->rows;
    a.cols = n->cols;
    a.x = n->x;
    a.res = n->residual;
    a.w = n->weight;
    a.h = n->h;
    a.y = n->y;
    a.ldx = n->ldx;
    a.ldr = n->ldr;
    a.ldh = n->ldh;
    a.ldy = n->ldy;
    a.q = codes_of(n->q);
    a.w_dtype = n->w_dtype;
    a.eps = n->eps;
    a.inv_cols = 1.0 / (double)n->cols;
    return done(launch_rms_norm(n->dtype, a, (hipStream_t)stream), "RMS norm launch");
}

int64_t opt_rms_norm_workspace(int64_t rows, int64_t cols)
{
    int rc;
    if ((rc = check_sides(rows, cols)) != OPT_OK) return rc;
    if (rows == 0 || cols == 0) return 0;
    if (cols > kMaxNormCols) return report(OPT_EUNSUPPORTED, "rows above %lld columns", (long long)kMaxNormCols);
    return norm_grad_groups(rows, cols) * cols * (int64_t)sizeof(float);
}

int opt_rms_norm_backward(const opt_norm_grad *n, void *stream)
{
    int rc;
    if (!n) return report(OPT_EINVAL, "the argument record is NULL");
    if ((rc = check_dtype(n->dtype, "dtype")) != OPT_OK) return rc;
    if ((rc = check_dtype(n->w_dtype, "w_dtype")) != OPT_OK) return rc;
    if ((rc = check_sides(n->rows, n->cols)) != OPT_OK) return rc;
    if (!(n->eps >= 0.0) || std::isinf(n->eps)) return report(OPT_EINVAL, "eps must be a non-negative number");
    if (n->accumulate != 0 && n->accumulate != 1) return report(OPT_EINVAL, "accumulate must be 0 or 1");
    if (n->cols == 0) return OPT_OK;
    if (n->cols > kMaxNormCols) return report(OPT_EUNSUPPORTED, "rows above %lld columns", (long long)kMaxNormCols);
    if (n->dweight && !at(n->dweight, 4)) return report(OPT_EALIGN, "dweight must be 4-byte aligned");
    if (n->rows > 0) {
        const size_t size = size_of(n->dtype);
        if ((rc = check_matrix("dy", n->dy, n->lddy, n->rows, n->cols, size)) != OPT_OK) return rc;
        if ((rc = check_matrix("h", n->h, n->ldh, n->rows, n->cols, size)) != OPT_OK) return rc;
        if ((rc = check_matrix("weight", n->weight, n->cols, 1, n->cols, size_of(n->w_dtype))) != OPT_OK) return rc;
        if (n->dh && (rc = check_matrix("dh", n->dh, n->lddh, n->rows, n->cols, size)) != OPT_OK) return rc;
        if ((rc = check_matrix("dx", n->dx, n->lddx, n->rows, n->cols, size)) != OPT_OK) return rc;
        if (n->dx == n->h) return report(OPT_EINVAL, "dx and h must be different matrices");
        if (n->dweight) {
            const int64_t need = norm_grad_groups(n->rows, n->cols) * n->cols * (int64_t)sizeof(float);
            if (!n->workspace) return report(OPT_EINVAL, "dweight needs a workspace");
            if (!at(n->workspace, 16)) return report(OPT_EALIGN, "the workspace must be 16-byte aligned");
            if (n->workspace_bytes < need)
                return report(OPT_EINVAL, "the workspace has %lld bytes of %lld", (long long)n->workspace_bytes, (long long)need);
        }
    } else if (!n->dweight) {
        return OPT_OK;
    }
    NormGradArgs a{};
    a.rows = n->rows;
    a.cols = n->cols;
    a.dy = n->dy;
    a.h = n->h;
    a.w = n->weight;
    a.dh = n->dh;
    a.dx = n->dx;
    a.lddy = n->lddy;
    a.ldh = n->ldh;
    a.lddh = n->lddh;
    a.lddx = n->lddx;
    a.part = n->dweight ? (float *)n->workspace : nullptr;
    a.w_dtype = n->w_dtype;
    a.eps = n->eps;
    a.inv_cols = 1.0 / (double)n->cols;
    return done(launch_rms_norm_grad(n->dtype, a, n->dweight, n->accumulate, (hipStream_t)stream), "RMS norm backward launch");
}

int opt_block_cast(const opt_cast *n, void *stream)
{
    int rc;
    if (!n) return report(OPT_EINVAL, "the argument record is NULL");
    if ((rc = check_dtype(n->dtype, "dtype")) != OPT_OK) return rc;
    if ((rc = check_sides(n->rows, n->cols)) != OPT_OK) return rc;
    if (n->block_rows != 1 && n->block_rows != kCodeBlock) return report(OPT_EINVAL, "block_rows must be 1 or 128");
    if (n->rows == 0 || n->cols == 0) return OPT_OK;
    if (!n->q.codes && !n->qt.codes) return report(OPT_EINVAL, "neither q nor qt is given");
    if ((rc = check_matrix("x", n->x, n->ldx, n->rows, n->cols, size_of(n->dtype))) != OPT_OK) return rc;
    if (n->q.codes && (rc = check_codes("q", n->q, n->rows, n->cols)) != OPT_OK) return rc;
    if (n->qt.codes && (rc = check_codes("qt", n->qt, n->cols, n->rows)) != OPT_OK) return rc;
    CastArgs a{};
    a.rows = n->rows;
    a.cols = n->cols;
    a.ldx = n->ldx;
    a.x = n->x;
    a.q = codes_of(n->q);
    a.qt = codes_of(n->qt);
    return done(launch_block_cast(n->dtype, a, n->block_rows == kCodeBlock, (hipStream_t)stream), "block cast launch");
}

int opt_block_matmul(const opt_product *n, void *stream)
{
    int rc;
    if (!n) return report(OPT_EINVAL, "the argument record is NULL");
    if ((rc = check_dtype(n->c_dtype, "c_dtype")) != OPT_OK) return rc;
    if ((rc = check_sides(n->m, n->n)) != OPT_OK) return rc;
    if (n->k < 0 || n->k >= kMaxSide || n->k % 16 != 0) return report(OPT_EINVAL, "k must be a multiple of 16 in [0, 2^31)");
    if (n->accumulate & ~(1 | OPT_CODE_PRODUCTS)) return report(OPT_EINVAL, "accumulate must be 0 or 1, with or without OPT_CODE_PRODUCTS");
    const int add = n->accumulate & 1;
    if (n->m == 0 || n->n == 0) return OPT_OK;
    if ((rc = check_matrix("c", n->c, n->ldc, n->m, n->n, size_of(n->c_dtype))) != OPT_OK) return rc;
    if (n->k > 0) {
        if ((rc = check_codes("a", n->a, n->m, n->k)) != OPT_OK) return rc;
        if ((rc = check_codes("b", n->b, n->n, n->k)) != OPT_OK) return rc;
    } else if (add) {
        return OPT_OK;
    }
    MatmulArgs a{};
    a.m = n->m;
    a.n = n->n;
    a.k = n->k;
    a.a = codes_of(n->a);
    a.b = codes_of(n->b);
    a.c = n->c;
    a.ldc = n->ldc;
    a.accumulate = add;
    a.exact = !(n->accumulate & OPT_CODE_PRODUCTS);
    return done(launch_block_matmul(n->c_dtype, a, (hipStream_t)stream), "block product launch");
}

int opt_gated_act(const opt_gate *n, void *stream)
{
    int rc;
    if (!n) return report(OPT_EINVAL, "the argument record is NULL");
    if ((rc = check_dtype(n->dtype, "dtype")) != OPT_OK) return rc;
    if ((rc = check_act(n->act)) != OPT_OK) return rc;
    if ((rc = check_sides(n->rows, n->cols)) != OPT_OK) return rc;
    if (n->rows == 0 || n->cols == 0) return OPT_OK;
    if (!n->y && !n->q.codes && !n->gate_q.codes && !n->up_q.codes) return report(OPT_EINVAL, "no output is given");
    const size_t size = size_of(n->dtype);
    if ((rc = check_matrix("gate", n->gate, n->ldg, n->rows, n->cols, size)) != OPT_OK) return rc;
    if ((rc = check_matrix("up", n->up, n->ldu, n->rows, n->cols, size)) != OPT_OK) return rc;
    if ((rc = check_more("y", n->y, n->ldy, n->rows, n->cols, size)) != OPT_OK) return rc;
    if ((rc = check_more("q", n->q, n->rows, n->cols)) != OPT_OK) return rc;
    if ((rc = check_more("gate_q", n->gate_q, n->rows, n->cols)) != OPT_OK) return rc;
    if ((rc = check_more("up_q", n->up_q, n->rows, n->cols)) != OPT_OK) return rc;
    if ((rc = check_apart({&n->q, &n->gate_q, &n->up_q})) != OPT_OK) return rc;
    if ((rc = check_over("y", n->y, n->ldy, n->gate, n->ldg, n->rows)) != OPT_OK) return rc;
    if ((rc = check_over("y", n->y, n->ldy, n->up, n->ldu, n->rows)) != OPT_OK) return rc;
    GateArgs a{};
    a.rows = n->rows;
    a.cols = n->cols;
    a.gate = n->gate;
    a.up = n->up;
    a.y = n->y;
    a.ldg = n->ldg;
    a.ldu = n->ldu;
    a.ldy = n->ldy;
    a.q = codes_of(n->q);
    a.gq = codes_of(n->gate_q);
    a.uq = codes_of(n->up_q);
    return done(launch_gated_act(n->dtype, n->act, a, (hipStream_t)stream), "gated activation launch");
}

int opt_gated_act_backward(const opt_gate_grad *n, void *stream)
{
    int rc;
    if (!n) return report(OPT_EINVAL, "the argument record is NULL");
    if ((rc = check_dtype(n->dtype, "dtype")) != OPT_OK) return rc;
    if ((rc = check_act(n->act)) != OPT_OK) return rc;
    if ((rc = check_sides(n->rows, n->cols)) != OPT_OK) return rc;
    if (n->rows == 0 || n->cols == 0) return OPT_OK;
    if (!n->dgate && !n->dup && !n->dgate_q.codes && !n->dup_q.codes && !n->dgate_t.codes && !n->dup_t.codes && !n->y_t.codes)
        return report(OPT_EINVAL, "no output is given");
    const size_t size = size_of(n->dtype);
    if ((rc = check_matrix("dy", n->dy, n->lddy, n->rows, n->cols, size)) != OPT_OK) return rc;
    if (n->gate || n->up) {
        if (n->gate_q.codes || n->up_q.codes) return report(OPT_EINVAL, "gate and up are given as matrices or as codes, not both");
        if ((rc = check_matrix("gate", n->gate, n->ldg, n->rows, n->cols, size)) != OPT_OK) return rc;
        if ((rc = check_matrix("up", n->up, n->ldu, n->rows, n->cols, size)) != OPT_OK) return rc;
    } else {
        if ((rc = check_codes("gate_q", n->gate_q, n->rows, n->cols)) != OPT_OK) return rc;
        if ((rc = check_codes("up_q", n->up_q, n->rows, n->cols)) != OPT_OK) return rc;
    }
    if ((rc = check_more("dgate", n->dgate, n->lddg, n->rows, n->cols, size)) != OPT_OK) return rc;
    if ((rc = check_more("dup", n->dup, n->lddu, n->rows, n->cols, size)) != OPT_OK) return rc;
    if (n->dgate && n->dgate == n->dup) return report(OPT_EINVAL, "dgate and dup must be different matrices");
    if ((rc = check_more("dgate_q", n->dgate_q, n->rows, n->cols)) != OPT_OK) return rc;
    if ((rc = check_more("dup_q", n->dup_q, n->rows, n->cols)) != OPT_OK) return rc;
    if ((rc = check_more("dgate_t", n->dgate_t, n->cols, n->rows)) != OPT_OK) return rc;
    if ((rc = check_more("dup_t", n->dup_t, n->cols, n->rows)) != OPT_OK) return rc;
    if ((rc = check_more("y_t", n->y_t, n->cols, n->rows)) != OPT_OK) return rc;
    if ((rc = check_apart({&n->dgate_q, &n->dup_q, &n->dgate_t, &n->dup_t, &n->y_t})) != OPT_OK) return rc;
    for (const opt_codes *in : {&n->gate_q, &n->up_q})
        if ((rc = check_apart({&n->dgate_t, &n->dup_t, &n->y_t, in})) != OPT_OK) return rc;
    const void *const in[3] = {n->dy, n->gate, n->up};
    const int64_t ld[3] = {n->lddy, n->ldg, n->ldu};
    for (int i = 0; i < 3; ++i) {
        if ((rc = check_over("dgate", n->dgate, n->lddg, in[i], ld[i], n->rows)) != OPT_OK) return rc;
        if ((rc = check_over("dup", n->dup, n->lddu, in[i], ld[i], n->rows)) != OPT_OK) return rc;
    }
    GateGradArgs a{};
    a.rows = n->rows;
    a.cols = n->cols;
    a.dy = n->dy;
    a.gate = n->gate;
    a.up = n->up;
    a.dgate = n->dgate;
    a.dup = n->dup;
    a.lddy = n->lddy;
    a.ldg = n->ldg;
    a.ldu = n->ldu;
    a.lddg = n->lddg;
    a.lddu = n->lddu;
    a.gq = codes_of(n->gate_q);
    a.uq = codes_of(n->up_q);
    a.dgq = codes_of(n->dgate_q);
    a.duq = codes_of(n->dup_q);
    a.dgt = codes_of(n->dgate_t);
    a.dut = codes_of(n->dup_t);
    a.yt = codes_of(n->y_t);
    return done(launch_gated_act_grad(n->dtype, n->act, a, (hipStream_t)stream), "gated activation backward launch");
}

int opt_block_restore(const opt_restore *n, void *stream)
{
    int rc;
    if (!n) return report(OPT_EINVAL, "the argument record is NULL");
    if ((rc = check_dtype(n->dtype, "dtype")) != OPT_OK) return rc;
    if ((rc = check_sides(n->rows, n->cols)) != OPT_OK) return rc;
    if (n->rows == 0 || n->cols == 0) return OPT_OK;
    if (!n->x && !n->qt.codes) return report(OPT_EINVAL, "neither x nor qt is given");
    if ((rc = check_codes("q", n->q, n->rows, n->cols)) != OPT_OK) return rc;
    if ((rc = check_more("x", n->x, n->ldx, n->rows, n->cols, size_of(n->dtype))) != OPT_OK) return rc;
    if ((rc = check_more("qt", n->qt, n->cols, n->rows)) != OPT_OK) return rc;
    if (n->qt.codes == n->q.codes) return report(OPT_EINVAL, "q and qt must be different matrices");
    RestoreArgs a{};
    a.rows = n->rows;
    a.cols = n->cols;
    a.q = codes_of(n->q);
    a.x = n->x;
    a.ldx = n->ldx;
    a.qt = codes_of(n->qt);
    return done(launch_block_restore(n->dtype, a, (hipStream_t)stream), "block restore launch");
}

int opt_head_norm(const opt_heads *n, void *stream)
{
    int rc;
    if (!n) return report(OPT_EINVAL, "the argument record is NULL");
    if ((rc = check_turn(n->tokens, n->dim, n->rot, n->dtype, n->w_dtype, n->interleaved, n->eps)) != OPT_OK) return rc;
    HeadArgs a{};
    int64_t heads = 0;
    for (int i = 0; i < 2; ++i) {
        const opt_head_set &s = i ? n->k : n->q;
        const char *const names[2][4] = {{"q", "q's x", "q's y", "q's weight"}, {"k", "k's x", "k's y", "k's weight"}};
        if ((rc = check_count(names[i][0], s.heads, n->tokens, s.codes.codes != nullptr)) != OPT_OK) return rc;
        heads += s.heads;
        if (s.heads == 0 || n->tokens == 0) continue;
        const size_t size = size_of(n->dtype);
        if ((rc = check_heads(names[i][1], s.x, s.x_token, s.x_head, n->tokens, s.heads, n->dim, size, false)) != OPT_OK) return rc;
        if ((rc = check_heads(names[i][2], s.y, s.y_token, s.y_head, n->tokens, s.heads, n->dim, size, true)) != OPT_OK) return rc;
        if ((rc = check_more(names[i][3], s.weight, n->dim, 1, n->dim, size_of(n->w_dtype))) != OPT_OK) return rc;
        if ((rc = check_more(names[i][0], s.codes, n->tokens * s.heads, n->dim)) != OPT_OK) return rc;
        if ((rc = check_over(names[i][2], s.y, s.y_token, s.y_head, s.x, s.x_token, s.x_head, n->tokens, s.heads)) != OPT_OK) return rc;
        HeadSet &d = a.s[i];
        d.heads = s.heads;
        d.x = s.x;
        d.w = s.weight;
        d.y = s.y;
        d.xt = s.x_token;
        d.xh = s.x_head;
        d.yt = s.y_token;
        d.yh = s.y_head;
        d.q = codes_of(s.codes);
    }
    if (n->tokens == 0 || heads == 0) return OPT_OK;
    if (n->q.heads && n->k.heads) {
        if (n->q.y == n->k.y) return report(OPT_EINVAL, "the two y must be different");
        if (n->q.y == n->k.x || n->k.y == n->q.x) return report(OPT_EINVAL, "y must not lie over the other set's x");
        if ((rc = check_apart({&n->q.codes, &n->k.codes})) != OPT_OK) return rc;
    }
    if ((rc = check_table(n->table, n->tokens, n->rot)) != OPT_OK) return rc;
    a.t = turn_of(n->tokens, n->dim, n->rot, n->w_dtype, n->interleaved, n->eps, n->table);
    return done(launch_head_norm(n->dtype, a, (hipStream_t)stream), "head norm launch");
}

int64_t opt_head_norm_workspace(int64_t tokens, int64_t heads_q, int64_t heads_k, int32_t dim)
{
    int rc;
    if (tokens < 0 || tokens >= kMaxSide) return report(OPT_EINVAL, "tokens must lie in [0, 2^31)");
    if ((rc = check_count("q", heads_q, tokens, false)) != OPT_OK) return rc;
    if ((rc = check_count("k", heads_k, tokens, false)) != OPT_OK) return rc;
    if (dim < 1) return report(OPT_EINVAL, "dim must be positive");
    if (dim > kMaxHeadDim) return report(OPT_EUNSUPPORTED, "heads above %d elements", kMaxHeadDim);
    if (tokens == 0 || heads_q + heads_k == 0) return 0;
    return head_grad_groups(tokens) * 2 * dim * (int64_t)sizeof(double);
}

int opt_head_norm_backward(const opt_heads_grad *n, void *stream)
{
    int rc;
    if (!n) return report(OPT_EINVAL, "the argument record is NULL");
    if ((rc = check_turn(n->tokens, n->dim, n->rot, n->dtype, n->w_dtype, n->interleaved, n->eps)) != OPT_OK) return rc;
    if (n->accumulate != 0 && n->accumulate != 1) return report(OPT_EINVAL, "accumulate must be 0 or 1");
    HeadGradArgs a{};
    int64_t heads = 0, coded = 0, plain = 0;
    for (int i = 0; i < 2; ++i) {
        const opt_head_grad_set &s = i ? n->k : n->q;
        const char *const names[2][5] = {{"q", "q's x", "q's dy", "q's dx", "q's weight"}, {"k", "k's x", "k's dy", "k's dx", "k's weight"}};
        if ((rc = check_count(names[i][0], s.heads, n->tokens, !s.x)) != OPT_OK) return rc;
        if (s.dweight && !at(s.dweight, 4)) return report(OPT_EALIGN, "dweight must be 4-byte aligned");
        heads += s.heads;
        if (s.heads == 0 || n->tokens == 0) continue;
        const size_t size = size_of(n->dtype);
        if (s.x && s.codes.codes) return report(OPT_EINVAL, "%s is given as a matrix or as codes, not both", names[i][1]);
        if (s.x) {
            ++plain;
            if ((rc = check_heads(names[i][1], s.x, s.x_token, s.x_head, n->tokens, s.heads, n->dim, size, false)) != OPT_OK) return rc;
        } else {
            ++coded;
            if ((rc = check_codes(names[i][1], s.codes, n->tokens * s.heads, n->dim)) != OPT_OK) return rc;
        }
        if ((rc = check_heads(names[i][2], s.dy, s.dy_token, s.dy_head, n->tokens, s.heads, n->dim, size, false)) != OPT_OK) return rc;
        if ((rc = check_heads(names[i][3], s.dx, s.dx_token, s.dx_head, n->tokens, s.heads, n->dim, size, true)) != OPT_OK) return rc;
        if (s.dx == s.x) return report(OPT_EINVAL, "dx and x must be different");
        if ((rc = check_over(names[i][3], s.dx, s.dx_token, s.dx_head, s.dy, s.dy_token, s.dy_head, n->tokens, s.heads)) != OPT_OK) return rc;
        if ((rc = check_more(names[i][4], s.weight, n->dim, 1, n->dim, size_of(n->w_dtype))) != OPT_OK) return rc;
        HeadGradSet &d = a.s[i];
        d.heads = s.heads;
        d.dy = s.dy;
        d.x = s.x;
        d.w = s.weight;
        d.dx = s.dx;
        d.dyt = s.dy_token;
        d.dyh = s.dy_head;
        d.xt = s.x_token;
        d.xh = s.x_head;
        d.dxt = s.dx_token;
        d.dxh = s.dx_head;
        d.q = codes_of(s.codes);
    }
    if (n->tokens > 0 && n->q.heads && n->k.heads) {
        if (n->q.dx == n->k.dx) return report(OPT_EINVAL, "the two dx must be different");
        if (n->q.dx == n->k.dy || n->q.dx == n->k.x || n->k.dx == n->q.dy || n->k.dx == n->q.x)
            return report(OPT_EINVAL, "dx must not lie over the other set's dy or x");
    }
    if (coded && plain) return report(OPT_EINVAL, "q and k are both given as matrices or both as codes");
    if (n->q.dweight && n->q.dweight == n->k.dweight) return report(OPT_EINVAL, "the two dweights must be different");
    const bool any = n->tokens > 0 && heads > 0, sums = n->q.dweight || n->k.dweight;
    if (any) {
        if ((rc = check_table(n->table, n->tokens, n->rot)) != OPT_OK) return rc;
        if (sums) {
            const int64_t need = head_grad_groups(n->tokens) * 2 * n->dim * (int64_t)sizeof(double);
            if (!n->workspace) return report(OPT_EINVAL, "dweight needs a workspace");
            if (!at(n->workspace, 16)) return report(OPT_EALIGN, "the workspace must be 16-byte aligned");
            if (n->workspace_bytes < need)
                return report(OPT_EINVAL, "the workspace has %lld bytes of %lld", (long long)n->workspace_bytes, (long long)need);
        }
    } else if (!sums) {
        return OPT_OK;
    }
    a.t = turn_of(n->tokens, n->dim, n->rot, n->w_dtype, n->interleaved, n->eps, n->table);
    a.part = any && sums ? (double *)n->workspace : nullptr;
    return done(launch_head_norm_grad(n->dtype, coded > 0, a, n->q.dweight, n->k.dweight, n->accumulate, (hipStream_t)stream),
                "head norm backward launch");
}

}  // extern "C"
