// opt_kernels_heads.hip -- the norm of queries and keys for each head with the
// rotation by position in the same pass, and its backward pass.
//
// Forward, for each head x of dim elements:  r = fl(1/sqrt(mean(x^2) + eps)),
// n = (x r) w, and the first rot elements turn in pairs (a, b) by the angle
// whose cosine c and sine s the position's row of the table holds:
// (a c - b s, b c + a s).  Backward: dn is dy turned the other way, g = dn w,
// k = mean(g x), dx = r (g - x r^2 k), dw = sum over tokens and heads of
// dn (x r).
//
// A head stays in the registers of L lanes, eight consecutive elements each; a
// wave holds 64/L heads (a unit) of one token and one of the two sets, and takes
// `per` units in turn, so that the token's angles are read once for them.
#include "opt_pass.h"

namespace optstep {

constexpr int kHeadThreads = 256;

// How a pair's other element is found.  kHalves: pairs (i, i + rot/2) with
// rot/2 and dim multiples of eight, so that the partners of a lane's eight are
// eight consecutive elements too.  kAny: everything else, element by element.
enum { kHalves = 0, kAny = 1 };

// A token's row of the table; 0 if its position has none.
__device__ __forceinline__ const float *table_row(const HeadTurn &t, int64_t token)
{
    int64_t p = token;
    if (t.positions) p = t.wide_positions ? gld<int64_t>((const int64_t *)t.positions + token) : (int64_t)gld<int32_t>((const int32_t *)t.positions + token);
    if (p < 0 || p >= t.table_rows) return nullptr;
    return t.table + p * t.ldt;
}

// cos and sin of the eight elements from c on, the sine with the sign of what
// the partner adds (BACK: turned the other way); 1 and 0 where nothing turns.
template <int MODE, bool BACK>
__device__ __forceinline__ void angles(const HeadTurn &t, const float *row, int c, float cs[8], float sn[8])
{
    const int h = t.rot / 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        cs[i] = 1.0f;
        sn[i] = 0.0f;
    }
    if (!row) return;
    if (MODE == kHalves) {
        if (c < t.rot) {
            const bool first = c < h;
            const float *p = row + (first ? c : c - h);
            load8<kP32>(p, 0, 8, cs);
            load8<kP32>(p + h, 0, 8, sn);
#pragma unroll
            for (int i = 0; i < 8; ++i) sn[i] = first != BACK ? -sn[i] : sn[i];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int e = c + i;
        if (e < t.rot) {
            const bool first = t.neighbours ? !(e & 1) : e < h;
            const int j = t.neighbours ? e >> 1 : first ? e : e - h;
            cs[i] = gld<float>(row + j);
            sn[i] = gld<float>(row + h + j);
            sn[i] = first != BACK ? -sn[i] : sn[i];
        }
    }
}

// The partners of the eight elements from c on, out of a head's row at p + at
// (elements that do not turn are their own).
template <int DT, int MODE>
__device__ __forceinline__ void partners(int dt, const HeadTurn &t, const void *p, int64_t at, int c, int cnt, const float own[8], float v[8])
{
    const int h = t.rot / 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = own[i];
    if (MODE == kHalves) {
        if (c < t.rot && cnt > 0) {
            const int64_t j = at + (c < h ? c + h : c - h);
            if (DT >= 0) load8<DT < 0 ? 0 : DT, true>(p, j, 8, v);
            else load8_any<true>(dt, p, j, 8, v);
        }
        return;
    }
    if (t.neighbours) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = own[i ^ 1];
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int e = c + i;
        if (e < t.rot && i < cnt) {
            const int64_t j = at + (e < h ? e + h : e - h);
            const int d = DT >= 0 ? DT : dt;
            if (d == kP32) v[i] = gld<float>((const float *)p + j);
            else {
                const uint32_t b = gld<uint16_t>((const uint16_t *)p + j);
                v[i] = d == kPBF16 ? bf16_lo(b) : f16_lo(b);
            }
        }
    }
}

// Largest over the lanes that share one 128-element block.
template <int L>
__device__ __forceinline__ uint32_t block_max_u32(uint32_t v)
{
    if (L >= 16) return row16_max_u32(v);
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));
    return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));
}

template <int L>
__device__ __forceinline__ double sum_squares(const float x[8])
{
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = __builtin_fma((double)x[i], (double)x[i], ss);
    return lanes_sum<L>(ss);
}

template <int DT, int L, int MODE>
__global__ __launch_bounds__(kHeadThreads) void head_norm_kernel(HeadArgs a, int per)
{
    constexpr int S = 64 / L;
    const HeadTurn &t = a.t;
    const int64_t u0 = (a.s[0].heads + S - 1) / S, units = u0 + (a.s[1].heads + S - 1) / S;
    const int64_t chunks = (units + per - 1) / per;
    const int lane = threadIdx.x % L, c = 8 * lane;
    const int cnt = left8(c, t.dim);
    const int64_t waves = t.tokens * chunks, step = (int64_t)gridDim.x * (kHeadThreads / 64);
    for (int64_t w = (int64_t)blockIdx.x * (kHeadThreads / 64) + threadIdx.x / 64; w < waves; w += step) {
        const int64_t token = w / chunks, first = (w % chunks) * per;
        const float *row = t.rot ? table_row(t, token) : nullptr;
        const bool lost = t.rot && !row;            // a position the table does not hold: NaN
        float cs[8], sn[8];
        angles<MODE, false>(t, row, c, cs, sn);
        for (int64_t u = first; u < first + per && u < units; ++u) {
            const int set = u >= u0;
            const HeadSet &s = a.s[set];
            const int64_t head = (u - (set ? u0 : 0)) * S + (threadIdx.x & 63) / L;
            const bool live = head < s.heads;
            const int n = live ? cnt : 0;
            float x[8], xp[8], wt[8], wp[8], y[8];
            const int64_t at = token * s.xt + head * s.xh;
            load8<DT, MODE == kHalves>(s.x, at + c, n, x);
            partners<DT, MODE>(0, t, s.x, at, c, n, x, xp);
            if (s.w) {
                load8_any<MODE == kHalves>(t.w_dtype, s.w, c, cnt, wt);
                partners<-1, MODE>(t.w_dtype, t, s.w, 0, c, cnt, wt, wp);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) wt[i] = wp[i] = 1.0f;
            }
            float r = (float)inverse_root(__builtin_fma(sum_squares<L>(x), t.inv_dim, t.eps));
            if (lost) r = bitsf(0x7FC00000u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float v = (x[i] * r) * wt[i], vp = (xp[i] * r) * wp[i];
                y[i] = c + i < t.rot ? v * cs[i] + vp * sn[i] : v;
            }
            store8<DT, MODE == kHalves>(s.y, token * s.yt + head * s.yh + c, n, y);
            if (s.q.codes) {
                uint32_t word;
                const u2 code = code_block(x, block_max_u32<L>(top8(x)), word);
                const int64_t line = token * s.heads + head;
                if (live && c < ((t.dim + 15) & ~15)) gst<u2>(s.q.codes + line * s.q.ld + c, code);
                if (n > 0 && (lane & 15) == 0) gst<uint8_t>(s.q.scales + (c / kCodeBlock) * s.q.lds + line, (uint8_t)(word >> 23));
            }
        }
    }
}

template <int DT, int L, int MODE, bool CODED>
__global__ __launch_bounds__(kHeadThreads) void head_norm_grad_kernel(HeadGradArgs a)
{
    constexpr int S = 64 / L;
    __shared__ float comb[4][2][L * 8];
    const HeadTurn &t = a.t;
    const int lane = threadIdx.x % L, c = 8 * lane;
    const int cnt = left8(c, t.dim);
    float dw[2][8] = {};
    const int64_t waves = t.tokens, step = (int64_t)gridDim.x * (kHeadThreads / 64);
    for (int64_t token = (int64_t)blockIdx.x * (kHeadThreads / 64) + threadIdx.x / 64; token < waves; token += step) {
        const float *row = t.rot ? table_row(t, token) : nullptr;
        const bool lost = t.rot && !row;
        float cs[8], sn[8];
        angles<MODE, true>(t, row, c, cs, sn);
#pragma unroll
        for (int set = 0; set < 2; ++set)
        for (int64_t head0 = 0; head0 < a.s[set].heads; head0 += S) {
            const HeadGradSet &s = a.s[set];
            const int64_t head = head0 + (threadIdx.x & 63) / L;
            const bool live = head < s.heads;
            const int n = live ? cnt : 0;
            float x[8], d[8], dp[8], wt[8], dx[8], g[8];
            const int64_t dat = token * s.dyt + head * s.dyh, line = token * s.heads + head;
            load8<DT, MODE == kHalves>(s.dy, dat + c, n, d);
            partners<DT, MODE>(0, t, s.dy, dat, c, n, d, dp);
            if (CODED) {
                u2 code = {0u, 0u};
                uint32_t byte = 127u;
                if (n > 0) {
                    code = gld<u2>(s.q.codes + line * s.q.ld + c);
                    byte = gld<uint8_t>(s.q.scales + (c / kCodeBlock) * s.q.lds + line);
                }
                decode8(code, byte, x);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = i < n ? x[i] : 0.0f;
            } else {
                load8<DT, MODE == kHalves>(s.x, token * s.xt + head * s.xh + c, n, x);
            }
            if (s.w) load8_any<MODE == kHalves>(t.w_dtype, s.w, c, cnt, wt);
            double sg = 0.0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (c + i < t.rot) d[i] = d[i] * cs[i] + dp[i] * sn[i];
                g[i] = s.w ? d[i] * wt[i] : d[i];
                sg = __builtin_fma((double)g[i], (double)x[i], sg);
            }
            float r = (float)inverse_root(__builtin_fma(sum_squares<L>(x), t.inv_dim, t.eps));
            if (lost) r = bitsf(0x7FC00000u);
            const float k = (float)((double)r * (double)r * (lanes_sum<L>(sg) * t.inv_dim));
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dx[i] = r * (g[i] - x[i] * k);
                if (live) dw[set][i] += d[i] * (x[i] * r);
            }
            store8<DT, MODE == kHalves>(s.dx, token * s.dxt + head * s.dxh + c, n, dx);
        }
    }
    if (!a.part) return;
    // the workgroup's sums: the heads of a wave by shuffles, then its waves through LDS, in a fixed order
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
#pragma unroll
            for (int off = L; off < 64; off <<= 1) dw[q][i] += __shfl_xor(dw[q][i], off, 64);
            if ((threadIdx.x & 63) < L) comb[threadIdx.x / 64][q][c + i] = dw[q][i];
        }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * t.dim; e += kHeadThreads) {
        const int q = e >= t.dim, j = e - q * t.dim;
        float v = comb[0][q][j];
        for (int w = 1; w < 4; ++w) v += comb[w][q][j];
        gst<float>(a.part + ((int64_t)blockIdx.x * 2 + q) * t.dim + j, v);
    }
}

// dw[c] (+)= sum over the groups' partials, in binary64 and a fixed order: 32
// columns a workgroup, 32 half-waves every 32nd group each.
__global__ __launch_bounds__(1024) void head_dw_kernel(const float *part, int64_t groups, int dim, float *dwq, float *dwk, int accumulate)
{
    __shared__ double s[32][32];
    const int lane = threadIdx.x % 32, rank = threadIdx.x / 32;
    const int e = (int)blockIdx.x * 32 + lane;
    double v = 0.0;
    if (e < 2 * dim) {
#pragma unroll 4
        for (int64_t g = rank; g < groups; g += 32) v += (double)gld<float>(part + g * 2 * dim + e);
    }
    s[rank][lane] = v;
    __syncthreads();
    if (rank == 0 && e < 2 * dim) {
        float *dw = e < dim ? dwq : dwk;
        if (!dw) return;
        const int j = e < dim ? e : e - dim;
        for (int i = 1; i < 32; ++i) v += s[i][lane];
        if (accumulate) v += (double)gld<float>(dw + j);
        gst<float>(dw + j, (float)v);
    }
}

// ---- launches --------------------------------------------------------------

static int head_lanes(int dim) { return dim <= 64 ? 8 : dim <= 128 ? 16 : dim <= 256 ? 32 : 64; }

static int64_t head_units(int64_t heads_q, int64_t heads_k, int dim)
{
    const int64_t per = 64 / head_lanes(dim);
    return (heads_q + per - 1) / per + (heads_k + per - 1) / per;
}

static bool by_halves(const HeadTurn &t) { return t.dim % 8 == 0 && (t.rot == 0 || (!t.neighbours && t.rot % 16 == 0)); }

int64_t head_grad_groups(int64_t tokens, int64_t heads_q, int64_t heads_k, int dim)
{
    const int64_t n = (tokens + kHeadThreads / 64 - 1) / (kHeadThreads / 64);
    return n < 512 ? n : 512;
}

template <int DT, int L>
static hipError_t launch_head_t(const HeadArgs &a, hipStream_t st)
{
    const int64_t units = head_units(a.s[0].heads, a.s[1].heads, a.t.dim);
    int64_t per = a.t.tokens * units / 8192;       // 8192 waves fill the chip
    per = per < 1 ? 1 : per > units ? units : per;
    const int64_t waves = a.t.tokens * ((units + per - 1) / per), want = (waves + kHeadThreads / 64 - 1) / (kHeadThreads / 64);
    const unsigned grid = (unsigned)(want < (1 << 20) ? want : 1 << 20);
    if (by_halves(a.t)) hipLaunchKernelGGL((head_norm_kernel<DT, L, kHalves>), dim3(grid), dim3(kHeadThreads), 0, st, a, (int)per);
    else hipLaunchKernelGGL((head_norm_kernel<DT, L, kAny>), dim3(grid), dim3(kHeadThreads), 0, st, a, (int)per);
    return hipGetLastError();
}

template <int DT, int L, bool CODED>
static hipError_t launch_head_grad_t(const HeadGradArgs &a, hipStream_t st)
{
    const unsigned grid = (unsigned)head_grad_groups(a.t.tokens, a.s[0].heads, a.s[1].heads, a.t.dim);
    if (by_halves(a.t)) hipLaunchKernelGGL((head_norm_grad_kernel<DT, L, kHalves, CODED>), dim3(grid), dim3(kHeadThreads), 0, st, a);
    else hipLaunchKernelGGL((head_norm_grad_kernel<DT, L, kAny, CODED>), dim3(grid), dim3(kHeadThreads), 0, st, a);
    return hipGetLastError();
}

template <int DT>
static hipError_t launch_head_dt(const HeadArgs &a, hipStream_t st)
{
    switch (head_lanes(a.t.dim)) {
    case 8: return launch_head_t<DT, 8>(a, st);
    case 16: return launch_head_t<DT, 16>(a, st);
    case 32: return launch_head_t<DT, 32>(a, st);
    default: return launch_head_t<DT, 64>(a, st);
    }
}

template <int DT, bool CODED>
static hipError_t launch_head_grad_dt(const HeadGradArgs &a, hipStream_t st)
{
    switch (head_lanes(a.t.dim)) {
    case 8: return launch_head_grad_t<DT, 8, CODED>(a, st);
    case 16: return launch_head_grad_t<DT, 16, CODED>(a, st);
    case 32: return launch_head_grad_t<DT, 32, CODED>(a, st);
    default: return launch_head_grad_t<DT, 64, CODED>(a, st);
    }
}

hipError_t launch_head_norm(int dt, const HeadArgs &a, hipStream_t st)
{
    if (dt == kP32) return launch_head_dt<kP32>(a, st);
    if (dt == kPBF16) return launch_head_dt<kPBF16>(a, st);
    return launch_head_dt<kPF16>(a, st);
}

hipError_t launch_head_norm_grad(int dt, int coded, const HeadGradArgs &a, float *dwq, float *dwk, int accumulate, hipStream_t st)
{
    hipError_t e = hipSuccess;
    const bool any = a.t.tokens > 0 && a.s[0].heads + a.s[1].heads > 0;
    if (any && coded) {
        e = dt == kP32 ? launch_head_grad_dt<kP32, true>(a, st) : dt == kPBF16 ? launch_head_grad_dt<kPBF16, true>(a, st) : launch_head_grad_dt<kPF16, true>(a, st);
    } else if (any) {
        e = dt == kP32 ? launch_head_grad_dt<kP32, false>(a, st) : dt == kPBF16 ? launch_head_grad_dt<kPBF16, false>(a, st) : launch_head_grad_dt<kPF16, false>(a, st);
    }
    if (e != hipSuccess || (!dwq && !dwk)) return e;
    const int64_t groups = any ? head_grad_groups(a.t.tokens, a.s[0].heads, a.s[1].heads, a.t.dim) : 0;
    hipLaunchKernelGGL(head_dw_kernel, dim3((unsigned)((2 * a.t.dim + 31) / 32)), dim3(1024), 0, st, (const float *)a.part, groups, a.t.dim, dwq, dwk,
                       accumulate);
    return hipGetLastError();
}

}  // namespace optstep
