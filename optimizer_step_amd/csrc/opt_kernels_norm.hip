// opt_kernels_norm.hip -- the root-mean-square norm with the residual's
// addition, an output in 16/32 bits and/or block-scaled 8-bit codes, and its
// backward pass.
//
// Forward, per row:  h = round(x + res),  r = fl(1 / sqrt(mean(h^2) + eps)),
// y = fl(fl(h * r) * w).  Backward:  g = dy * w,  c = mean(g * h),
// dx = r * (g - h * (r^2 c)) [+ dh],  dw = sum over rows of dy * (h * r).
//
// Both are bound by HBM: every matrix crosses it once (8192 x 4096 bf16: with
// the residual and codes 45 us for 237 MB, 5.2 TB/s; backward with the
// residual's gradient 55.5 us for 268 MB, of which the weight's gradient 5).
// A row stays in the registers of `LANES` lanes, eight consecutive elements (16 bytes of 16-bit
// words) a lane at a time, so that a 128-column block is one 16-lane DPP row
// and its largest magnitude takes four DPP steps.  Squares are summed in
// binary64, whose rate is half of binary32's here and leaves the kernel bound
// by memory: r, rounded to binary32, then hardly ever depends on the order of
// the sum (only where a few binary64 units straddle a rounding border).
#include "opt_pass.h"

namespace optstep {

constexpr int norm_threads(int lanes) { return lanes < 256 ? 256 : lanes; }

// The sums of a row over its LANES lanes, in every lane.  Waves meet in `slot`
// (N doubles a wave): one barrier, as consecutive calls take alternate slots.
template <int LANES, int N>
__device__ __forceinline__ void row_sums(double (&v)[N], double (*slot)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lanes_sum<LANES>(v[i]);
    if (LANES > 64) {
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int i = 0; i < N; ++i) slot[threadIdx.x >> 6][i] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = slot[0][i];
#pragma unroll
        for (int w = 1; w < LANES / 64; ++w)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += slot[w][i];
    }
}

// EIGHTS: rows of a multiple of eight elements, without the code for single
// ones (8192 x 4096 bf16 to codes 25.2 us, with it 26.9).
//
// h stays in its stored form between the sum and the result: for 16-bit types
// half the registers.  Stores carry the non-temporal hint: 51 -> 46 us at
// 8192 x 4096 bf16 with a residual and codes; on the loads it costs as much.
template <int DT, int LANES, int VECS, bool EIGHTS>
__global__ __launch_bounds__(norm_threads(LANES)) void rms_norm_kernel(NormArgs a)
{
    constexpr int kRows = norm_threads(LANES) / LANES;   // rows a workgroup holds at once
    __shared__ double slot[2][16][1];
    const int lane = threadIdx.x % LANES;
    int turn = 0;
    for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < a.rows; r0 += (int64_t)gridDim.x * kRows, turn ^= 1) {
        const int64_t row = r0 + threadIdx.x / LANES;
        const bool live = row < a.rows;
        Raw<DT> h[VECS];
        double ss[1] = {0.0};
#pragma unroll
        for (int j = 0; j < VECS; ++j) {
            const int64_t c = 8 * (int64_t)(lane + j * LANES);
            h[j] = load_raw<DT, EIGHTS>(a.x, row * a.ldx + c, live ? left8(c, a.cols) : 0);
        }
        if (a.res) {
            Raw<DT> t[VECS];
#pragma unroll
            for (int j = 0; j < VECS; ++j) {
                const int64_t c = 8 * (int64_t)(lane + j * LANES);
                t[j] = load_raw<DT, EIGHTS>(a.res, row * a.ldr + c, live ? left8(c, a.cols) : 0);
            }
#pragma unroll
            for (int j = 0; j < VECS; ++j) {
                float u[8], v[8];
                unpack_raw<DT>(h[j], u);
                unpack_raw<DT>(t[j], v);
#pragma unroll
                for (int i = 0; i < 8; ++i) u[i] = u[i] + v[i];
                h[j] = pack_raw<DT>(u);
            }
        }
#pragma unroll
        for (int j = 0; j < VECS; ++j) {
            const int64_t c = 8 * (int64_t)(lane + j * LANES);
            if (a.h) store_raw<DT, EIGHTS, true>(a.h, row * a.ldh + c, live ? left8(c, a.cols) : 0, h[j]);
            float u[8];
            unpack_raw<DT>(h[j], u);
#pragma unroll
            for (int i = 0; i < 8; ++i) ss[0] = __builtin_fma((double)u[i], (double)u[i], ss[0]);
        }
        row_sums<LANES, 1>(ss, slot[turn]);
        const float r = (float)inverse_root(__builtin_fma(ss[0], a.inv_cols, a.eps));
#pragma unroll
        for (int j = 0; j < VECS; ++j) {
            const int64_t c = 8 * (int64_t)(lane + j * LANES);
            const int cnt = live ? left8(c, a.cols) : 0;
            float w[8], u[8], y[8];
            load8_any<EIGHTS>(a.w_dtype, a.w, c, left8(c, a.cols), w);
            unpack_raw<DT>(h[j], u);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = i < cnt ? (u[i] * r) * w[i] : 0.0f;
            if (a.y) store8<DT, EIGHTS, true>(a.y, row * a.ldy + c, cnt, y);
            if (a.q.codes) {
                const uint32_t byte = block_scale(row16_max_u32(abs_max8(y)));
                const u2 code = encode8(y, byte);
                if (live && c < ((a.cols + 15) & ~(int64_t)15)) sst<u2>(a.q.codes + row * a.q.ld + c, code);
                if (cnt > 0 && (lane & 15) == 0) gst<uint8_t>(a.q.scales + (c / kCodeBlock) * a.q.lds + row, (uint8_t)byte);
            }
        }
    }
}

// A row of the backward pass as it is stored.
template <int DT, int VECS>
struct GradRow { Raw<DT> h[VECS], dy[VECS], dh[VECS]; };

template <int DT, int LANES, int VECS, bool EIGHTS>
__device__ __forceinline__ void load_row(const NormGradArgs &a, int64_t row, GradRow<DT, VECS> &g)
{
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
        const int64_t c = 8 * (int64_t)(threadIdx.x % LANES + j * LANES);
        const int cnt = row < a.rows ? left8(c, a.cols) : 0;
        g.h[j] = load_raw<DT, EIGHTS>(a.h, row * a.ldh + c, cnt);
        g.dy[j] = load_raw<DT, EIGHTS>(a.dy, row * a.lddy + c, cnt);
        if (a.dh) g.dh[j] = load_raw<DT, EIGHTS>(a.dh, row * a.lddh + c, cnt);
    }
}

// A workgroup takes every gridDim.x-th row (or group of rows) and keeps its
// columns' sums of dy * (h * r) in registers; where two rows fit there (not in
// the 128 registers of 1024 lanes), the next one is on its way while this one's
// sums are formed.  1024 lanes spill: above 16384 columns 212 to 535 registers
// (250 to 1634 where single elements are handled too), 1.5 TB/s at 1024 x 32768
// bf16; for 8193 to 16384 columns 6 or 8 (2 to 17; fp32 362), 4.2 TB/s at
// 2048 x 16384 and 3.0 at 2048 x 16383.
template <int DT, int LANES, int VECS, bool EIGHTS>
__global__ __launch_bounds__(norm_threads(LANES)) void rms_norm_grad_kernel(NormGradArgs a)
{
    constexpr int kRows = norm_threads(LANES) / LANES;
    constexpr bool kAhead = LANES < 1024 && VECS * (int)sizeof(typename Elem<DT>::T) <= 8;
    __shared__ double slot[2][16][2];
    __shared__ float comb[LANES < 256 ? 256 * 8 : 1];
    const int lane = threadIdx.x % LANES;
    const int64_t step = (int64_t)gridDim.x * kRows;
    constexpr bool kKeep = VECS <= 2;           // the weight stays in registers
    float dw[VECS][8] = {}, w[kKeep ? VECS : 1][8];
    if (kKeep)
#pragma unroll
        for (int j = 0; j < VECS; ++j) {
            const int64_t c = 8 * (int64_t)(lane + j * LANES);
            load8_any<EIGHTS>(a.w_dtype, a.w, c, left8(c, a.cols), w[j * kKeep]);
        }
    // one row (or group of rows); `g` holds it, `next` takes the one after it
    auto one = [&](int64_t row, GradRow<DT, VECS> &g, GradRow<DT, VECS> &next, int turn) {
        const bool live = row < a.rows;
        if (kAhead) load_row<DT, LANES, VECS, EIGHTS>(a, row + step, next);
        double s[2] = {0.0, 0.0};
#pragma unroll
        for (int j = 0; j < VECS; ++j) {
            const int64_t c = 8 * (int64_t)(lane + j * LANES);
            float h[8], dy[8];
            if (!kKeep) load8_any<EIGHTS>(a.w_dtype, a.w, c, left8(c, a.cols), w[0]);
            unpack_raw<DT>(g.h[j], h);
            unpack_raw<DT>(g.dy[j], dy);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const double hd = (double)h[i];
                s[0] = __builtin_fma(hd, hd, s[0]);
                s[1] = __builtin_fma((double)(dy[i] * w[j * kKeep][i]), hd, s[1]);
            }
        }
        row_sums<LANES, 2>(s, slot[turn]);
        const float r = (float)inverse_root(__builtin_fma(s[0], a.inv_cols, a.eps));
        const float k = (float)((double)r * (double)r * (s[1] * a.inv_cols));
#pragma unroll
        for (int j = 0; j < VECS; ++j) {
            const int64_t c = 8 * (int64_t)(lane + j * LANES);
            const int cnt = live ? left8(c, a.cols) : 0;
            float h[8], dy[8], dx[8];
            if (!kKeep) load8_any<EIGHTS>(a.w_dtype, a.w, c, left8(c, a.cols), w[0]);
            unpack_raw<DT>(g.h[j], h);
            unpack_raw<DT>(g.dy[j], dy);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dx[i] = r * (dy[i] * w[j * kKeep][i] - h[i] * k);
                if (live) dw[j][i] += dy[i] * (h[i] * r);
            }
            if (a.dh) {
                float t[8];
                unpack_raw<DT>(g.dh[j], t);
#pragma unroll
                for (int i = 0; i < 8; ++i) dx[i] = dx[i] + t[i];
            }
            store8<DT, EIGHTS, true>(a.dx, row * a.lddx + c, cnt, dx);
        }
    };
    int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / LANES, r0 = (int64_t)blockIdx.x * kRows;
    GradRow<DT, VECS> g0, g1;
    load_row<DT, LANES, VECS, EIGHTS>(a, row, g0);
    while (r0 < a.rows) {
        one(row, g0, g1, 0);
        row += step;
        r0 += step;
        if (r0 >= a.rows) break;
        if (!kAhead) load_row<DT, LANES, VECS, EIGHTS>(a, row, g0);
        one(row, kAhead ? g1 : g0, g0, 1);
        row += step;
        r0 += step;
        if (!kAhead && r0 < a.rows) load_row<DT, LANES, VECS, EIGHTS>(a, row, g0);
    }
    if (!a.part) return;
    // the workgroup's partial sums: rows of one wave by shuffles, then waves
    // through LDS, in a fixed order
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
        const int64_t c = 8 * (int64_t)(lane + j * LANES);
        if (LANES < 256) {
#pragma unroll
            for (int off = LANES; off < 64; off <<= 1)
#pragma unroll
                for (int i = 0; i < 8; ++i) dw[j][i] += __shfl_xor(dw[j][i], off, 64);
            constexpr int L = LANES < 64 ? LANES : 64;
            __syncthreads();
            if ((threadIdx.x & 63) < L)
                for (int i = 0; i < 8; ++i) comb[((threadIdx.x >> 6) * L + (threadIdx.x & 63)) * 8 + i] = dw[j][i];
            __syncthreads();
            if (threadIdx.x < L) {
                float v[8];
                for (int i = 0; i < 8; ++i) {
                    v[i] = comb[threadIdx.x * 8 + i];
                    for (int s = 1; s < 4; ++s) v[i] += comb[(s * L + threadIdx.x) * 8 + i];
                }
                store8<kP32>(a.part, (int64_t)blockIdx.x * a.cols + c, left8(c, a.cols), v);
            }
        } else {
            store8<kP32>(a.part, (int64_t)blockIdx.x * a.cols + c, left8(c, a.cols), dw[j]);
        }
    }
}

// dw[c] (+)= sum over the groups' partials, in binary64 and a fixed order: 32
// columns a workgroup, 32 half-waves every 32nd group each.
constexpr int kDwCols = 32;

__global__ __launch_bounds__(1024) void norm_dw_kernel(const float *part, int64_t groups, int64_t cols, float *dw, int accumulate)
{
    __shared__ double s[32][kDwCols];
    const int lane = threadIdx.x % kDwCols, rank = threadIdx.x / kDwCols;
    const int64_t c = (int64_t)blockIdx.x * kDwCols + lane;
    double v = 0.0;
    if (c < cols) {
#pragma unroll 8
        for (int64_t g = rank; g < groups; g += 32) v += (double)gld<float>(part + g * cols + c);
    }
    s[rank][lane] = v;
    __syncthreads();
    if (rank == 0 && c < cols) {
        for (int i = 1; i < 32; ++i) v += s[i][lane];
        if (accumulate) v += (double)gld<float>(dw + c);
        gst<float>(dw + c, (float)v);
    }
}

// A workgroup of 256 holds a row of 2048 to 8192 columns: a wave alone (no
// barrier, 32 KB in flight) measured 54 us against 45 forward and 97 against 61
// backward at 8192 x 4096.
NormShape norm_shape(int64_t cols)
{
    const int64_t v = (cols + 7) / 8;                 // groups of eight in a row
    NormShape s;
    s.lanes = v <= 64 ? 16 : v <= 256 ? 64 : v <= 1024 ? 256 : 1024;
    s.vecs = 1;
    while ((int64_t)s.lanes * s.vecs < v) s.vecs *= 2;
    return s;
}

int64_t norm_grad_groups(int64_t rows, int64_t cols)
{
    const NormShape s = norm_shape(cols);
    const int64_t per = s.lanes < 256 ? 256 / s.lanes : 1;
    const int64_t n = (rows + per - 1) / per;
    const int64_t most = s.lanes == 1024 ? 256 : 512;   // two workgroups a compute unit; 768 measured 57.3 us, 1024 61.5 against 55.5
    return n < most ? n : most;
}

#define NORM_SHAPES(X) X(16, 1) X(16, 2) X(16, 4) X(64, 2) X(64, 4) X(256, 2) X(256, 4) X(1024, 2) X(1024, 4)

template <int DT>
static hipError_t launch_norm_t(const NormArgs &a, hipStream_t st)
{
    const NormShape s = norm_shape(a.cols);
    const int64_t per = s.lanes < 256 ? 256 / s.lanes : 1;
    const int64_t want = (a.rows + per - 1) / per;
    const unsigned grid = (unsigned)(want < (1 << 20) ? want : 1 << 20);
#define X(L, V) \
    if (s.lanes == L && s.vecs == V) { \
        if (a.cols % 8 == 0) hipLaunchKernelGGL((rms_norm_kernel<DT, L, V, true>), dim3(grid), dim3(norm_threads(L)), 0, st, a); \
        else hipLaunchKernelGGL((rms_norm_kernel<DT, L, V, false>), dim3(grid), dim3(norm_threads(L)), 0, st, a); \
        return hipGetLastError(); \
    }
    NORM_SHAPES(X)
#undef X
    return hipErrorInvalidValue;
}

template <int DT>
static hipError_t launch_norm_grad_t(const NormGradArgs &a, hipStream_t st)
{
    const NormShape s = norm_shape(a.cols);
    const unsigned grid = (unsigned)norm_grad_groups(a.rows, a.cols);
#define X(L, V) \
    if (s.lanes == L && s.vecs == V) { \
        if (a.cols % 8 == 0) hipLaunchKernelGGL((rms_norm_grad_kernel<DT, L, V, true>), dim3(grid), dim3(norm_threads(L)), 0, st, a); \
        else hipLaunchKernelGGL((rms_norm_grad_kernel<DT, L, V, false>), dim3(grid), dim3(norm_threads(L)), 0, st, a); \
        return hipGetLastError(); \
    }
    NORM_SHAPES(X)
#undef X
    return hipErrorInvalidValue;
}

hipError_t launch_rms_norm(int dt, const NormArgs &a, hipStream_t st)
{
    if (dt == kP32) return launch_norm_t<kP32>(a, st);
    if (dt == kPBF16) return launch_norm_t<kPBF16>(a, st);
    return launch_norm_t<kPF16>(a, st);
}

hipError_t launch_rms_norm_grad(int dt, const NormGradArgs &a, float *dw, int accumulate, hipStream_t st)
{
    hipError_t e = hipSuccess;
    if (a.rows > 0) e = dt == kP32 ? launch_norm_grad_t<kP32>(a, st) : dt == kPBF16 ? launch_norm_grad_t<kPBF16>(a, st)
                                                                                    : launch_norm_grad_t<kPF16>(a, st);
    if (e != hipSuccess || !dw) return e;
    const int64_t groups = a.rows > 0 ? norm_grad_groups(a.rows, a.cols) : 0;
    hipLaunchKernelGGL(norm_dw_kernel, dim3((unsigned)((a.cols + kDwCols - 1) / kDwCols)), dim3(1024), 0, st, (const float *)a.part, groups,
                       a.cols, dw, accumulate);
    return hipGetLastError();
}

}  // namespace optstep
