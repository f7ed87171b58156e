// opt_kernels_norm.hip -- the root-mean-square norm with the residual's
// addition, an output in 16/32 bits and/or block-scaled 8-bit codes, and its
// backward pass.
//
// Forward, per row:  h = round(x + res),  r = fl(1 / sqrt(mean(h^2) + eps)),
// y = fl(fl(h * r) * w).  Backward:  g = dy * w,  c = mean(g * h),
// dx = r * (g - h * (r^2 c)) [+ dh],  dw = sum over rows of dy * (h * r).
//
// Both are bound by HBM: every matrix crosses it once.  A row stays in the
// registers of `LANES` lanes, eight consecutive elements (16 bytes of 16-bit
// words) a lane at a time, so that a 128-column block is one 16-lane DPP row
// and its largest magnitude takes four DPP steps.  Squares are summed in
// binary64, whose rate is half of binary32's here and leaves the kernel bound
// by memory: r is then the same bits in whatever order the sum ran.
#include "opt_pass.h"

namespace optstep {

// Sum over the LANES lanes of a row, the same bits in every lane; `slot` is
// LDS scratch of a double per wave, used twice per call site at most.
template <int LANES>
__device__ __forceinline__ double row_sum(double v, double *slot)
{
#pragma unroll
    for (int off = 1; off < (LANES < 64 ? LANES : 64); off <<= 1) v += __shfl_xor(v, off, 64);
    if (LANES > 64) {
        __syncthreads();
        if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0;
        for (int w = 0; w < LANES / 64; ++w) v += slot[w];
    }
    return v;
}

constexpr int norm_threads(int lanes) { return lanes < 256 ? 256 : lanes; }

template <int DT, int LANES, int VECS>
__global__ __launch_bounds__(norm_threads(LANES)) void rms_norm_kernel(NormArgs a)
{
    constexpr int kRows = norm_threads(LANES) / LANES;   // rows a workgroup holds at once
    __shared__ double slot[16];
    const int lane = threadIdx.x % LANES;
    for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < a.rows; r0 += (int64_t)gridDim.x * kRows) {
        const int64_t row = r0 + threadIdx.x / LANES;
        const bool live = row < a.rows;
        float h[VECS][8];
        double ss = 0.0;
#pragma unroll
        for (int j = 0; j < VECS; ++j) {
            const int64_t c = 8 * (int64_t)(lane + j * LANES);
            const int cnt = live ? left8(c, a.cols) : 0;
            load8<DT>(a.x, row * a.ldx + c, cnt, h[j]);
            if (a.res) {
                float t[8];
                load8<DT>(a.res, row * a.ldr + c, cnt, t);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[j][i] = stored<DT>(h[j][i] + t[i]);
            }
            if (a.h) store8<DT>(a.h, row * a.ldh + c, cnt, h[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = __builtin_fma((double)h[j][i], (double)h[j][i], ss);
        }
        ss = row_sum<LANES>(ss, slot);
        const float r = (float)(1.0 / sqrt(ss / (double)a.cols + a.eps));
#pragma unroll
        for (int j = 0; j < VECS; ++j) {
            const int64_t c = 8 * (int64_t)(lane + j * LANES);
            const int cnt = live ? left8(c, a.cols) : 0;
            float w[8], y[8];
            load8_any(a.w_dtype, a.w, c, left8(c, a.cols), w);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = i < cnt ? (h[j][i] * r) * w[i] : 0.0f;
            if (a.y) store8<DT>(a.y, row * a.ldy + c, cnt, y);
            if (a.q.codes) {
                const uint32_t byte = block_scale(row16_max_u32(abs_max8(y)));
                const u2 code = encode8(y, byte);
                if (live && c < ((a.cols + 15) & ~(int64_t)15)) gst<u2>(a.q.codes + row * a.q.ld + c, code);
                if (cnt > 0 && (lane & 15) == 0) gst<uint8_t>(a.q.scales + (c / kCodeBlock) * a.q.lds + row, (uint8_t)byte);
            }
        }
    }
}

template <int DT, int LANES, int VECS>
__global__ __launch_bounds__(norm_threads(LANES)) void rms_norm_grad_kernel(NormGradArgs a)
{
    constexpr int kRows = norm_threads(LANES) / LANES;
    __shared__ double slot[16], slot2[16];
    __shared__ float comb[LANES < 256 ? 256 * 8 : 1];
    const int lane = threadIdx.x % LANES;
    float dw[VECS][8] = {};
    for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < a.rows; r0 += (int64_t)gridDim.x * kRows) {
        const int64_t row = r0 + threadIdx.x / LANES;
        const bool live = row < a.rows;
        float h[VECS][8], dy[VECS][8];
        double ss = 0.0, gh = 0.0;
#pragma unroll
        for (int j = 0; j < VECS; ++j) {
            const int64_t c = 8 * (int64_t)(lane + j * LANES);
            const int cnt = live ? left8(c, a.cols) : 0;
            float w[8];
            load8<DT>(a.h, row * a.ldh + c, cnt, h[j]);
            load8<DT>(a.dy, row * a.lddy + c, cnt, dy[j]);
            load8_any(a.w_dtype, a.w, c, left8(c, a.cols), w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ss = __builtin_fma((double)h[j][i], (double)h[j][i], ss);
                gh = __builtin_fma((double)(dy[j][i] * w[i]), (double)h[j][i], gh);
            }
        }
        ss = row_sum<LANES>(ss, slot);
        gh = row_sum<LANES>(gh, slot2);
        const float r = (float)(1.0 / sqrt(ss / (double)a.cols + a.eps));
        const float k = (float)((double)r * (double)r * (gh / (double)a.cols));
#pragma unroll
        for (int j = 0; j < VECS; ++j) {
            const int64_t c = 8 * (int64_t)(lane + j * LANES);
            const int cnt = live ? left8(c, a.cols) : 0;
            float w[8], t[8] = {}, dx[8];
            load8_any(a.w_dtype, a.w, c, left8(c, a.cols), w);
            if (a.dh) load8<DT>(a.dh, row * a.lddh + c, cnt, t);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dx[i] = r * (dy[j][i] * w[i] - h[j][i] * k);
                if (a.dh) dx[i] = dx[i] + t[i];
                if (live) dw[j][i] += dy[j][i] * (h[j][i] * r);
            }
            store8<DT>(a.dx, row * a.lddx + c, cnt, dx);
        }
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

// dw[c] (+)= sum over the groups' partials, in binary64 and a fixed order: 64
// columns a workgroup, four waves a quarter of the groups each.
__global__ __launch_bounds__(256) void norm_dw_kernel(const float *part, int64_t groups, int64_t cols, float *dw, int accumulate)
{
    __shared__ double s[4][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
    const int64_t c = (int64_t)blockIdx.x * 64 + lane;
    double v = 0.0;
    if (c < cols)
        for (int64_t g = wave; g < groups; g += 4) v += (double)gld<float>(part + g * cols + c);
    s[wave][lane] = v;
    __syncthreads();
    if (wave == 0 && c < cols) {
        v = ((s[0][lane] + s[1][lane]) + s[2][lane]) + s[3][lane];
        if (accumulate) v += (double)gld<float>(dw + c);
        gst<float>(dw + c, (float)v);
    }
}

NormShape norm_shape(int64_t cols)
{
    const int64_t v = (cols + 7) / 8;                 // groups of eight in a row
    NormShape s;
    s.lanes = v <= 64 ? 16 : v <= 256 ? 64 : v <= 2048 ? 256 : 1024;
    s.vecs = 1;
    while ((int64_t)s.lanes * s.vecs < v) s.vecs *= 2;
    return s;
}

int64_t norm_grad_groups(int64_t rows, int64_t cols)
{
    const NormShape s = norm_shape(cols);
    const int64_t per = s.lanes < 256 ? 256 / s.lanes : 1;
    const int64_t n = (rows + per - 1) / per;
    const int64_t most = s.lanes == 1024 ? 256 : 1024;
    return n < most ? n : most;
}

#define NORM_SHAPES(X) X(16, 1) X(16, 2) X(16, 4) X(64, 2) X(64, 4) X(256, 2) X(256, 4) X(256, 8) X(1024, 4)

template <int DT>
static hipError_t launch_norm_t(const NormArgs &a, hipStream_t st)
{
    const NormShape s = norm_shape(a.cols);
    const int64_t per = s.lanes < 256 ? 256 / s.lanes : 1;
    const int64_t want = (a.rows + per - 1) / per;
    const unsigned grid = (unsigned)(want < (1 << 20) ? want : 1 << 20);
#define X(L, V) \
    if (s.lanes == L && s.vecs == V) { \
        hipLaunchKernelGGL((rms_norm_kernel<DT, L, V>), dim3(grid), dim3(norm_threads(L)), 0, st, a); \
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
        hipLaunchKernelGGL((rms_norm_grad_kernel<DT, L, V>), dim3(grid), dim3(norm_threads(L)), 0, st, a); \
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
    hipLaunchKernelGGL(norm_dw_kernel, dim3((unsigned)((a.cols + 63) / 64)), dim3(256), 0, st, (const float *)a.part, groups,
                       a.cols, dw, accumulate);
    return hipGetLastError();
}

}  // namespace optstep
