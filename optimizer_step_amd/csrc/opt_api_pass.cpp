// opt_api_pass.cpp -- the C ABI of the training-pass operators: argument
// checks and launches.  Nothing here holds state: what an operator needs
// besides its tensors the caller passes.
#include <hip/hip_runtime.h>

#include <cmath>

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

}  // extern "C"
