// opt_kernels_gate.hip -- the gated activation y = s(gate) * up with its
// inputs kept as block-coded 8-bit checkpoints, its backward pass from those
// codes or from the matrices, and the restoring of a coded matrix.
//
// s(x) = x sigma(p(x)), sigma the logistic function: p(x) = x is SiLU, p(x) =
// 2 sqrt(2/pi) (x + 0.044715 x^3) the tanh form of GELU (0.5 (1 + tanh(z)) =
// sigma(2 z)).  s'(x) = sigma (1 + x (1 - sigma) p'(x)).
#include "opt_pass.h"

namespace optstep {

// sigma(p) and 1 - sigma(p), each to a few binary32 units of itself: both come
// from e = exp(-|p|) <= 1, so neither overflows nor cancels.  FINE: the rounding
// of |p| log2(e), which exp2 would make relative |p| 2^-24 of e, is carried
// along (|p| held at 256, where e is 0, so that it is finite); 16-bit and 8-bit
// results do not see it.  A NaN p may give any values: its x makes them NaN.
template <bool FINE>
__device__ __forceinline__ void logistic(float p, float &sig, float &rest)
{
    const float a = FINE ? __builtin_fminf(__builtin_fabsf(p), 256.0f) : __builtin_fabsf(p);
    const float t = a * -1.44269504f;
    float e = __builtin_amdgcn_exp2f(t);
    if (FINE) {
        // -a log2(e) = t + (its rounding + a times what the constant lacks)
        const float lo = __builtin_fmaf(a, -1.92596299e-8f, __builtin_fmaf(a, -1.44269504f, -t));
        e = __builtin_fmaf(e * 0.693147181f, lo, e);
    }
    const float big = __builtin_amdgcn_rcpf(1.0f + e), small = e * big;
    sig = p >= 0.0f ? big : small;
    rest = p >= 0.0f ? small : big;
}

// p(x) and p'(x).  GELU: beyond |x| = 16 exp(-|p|) is 0 in binary32, so x is
// held there and its cube stays finite.
template <int ACT>
__device__ __forceinline__ void inner(float x, float &p, float &dp)
{
    if (ACT == kActSilu) {
        p = x;
        dp = 1.0f;
        return;
    }
    constexpr float k = 1.59576912f, kc = 0.0713548163f;     // 2 sqrt(2/pi), the same times 0.044715
    const float c = __builtin_amdgcn_fmed3f(x, -16.0f, 16.0f);
    const float c2 = c * c;
    p = c * __builtin_fmaf(c2, kc, k);
    dp = __builtin_fmaf(c2, 3.0f * kc, k);
}

template <int ACT, bool FINE>
__device__ __forceinline__ float act(float x)
{
    float p, dp, sig, rest;
    inner<ACT>(x, p, dp);
    logistic<FINE>(p, sig, rest);
    return x * sig;
}

template <int ACT, bool FINE>
__device__ __forceinline__ void act_slope(float x, float &s, float &slope)
{
    float p, dp, sig, rest;
    inner<ACT>(x, p, dp);
    logistic<FINE>(p, sig, rest);
    s = x * sig;
    slope = __builtin_fmaf(s * rest, dp, sig);
}

// One row's block of 128 columns by 16 lanes: codes and the scale's byte.
__device__ __forceinline__ void put_block(const Codes &q, int64_t row, int64_t c, bool live, int64_t cols16, const float v[8])
{
    const uint32_t byte = block_scale(row16_max_u32(abs_max8(v)));
    const u2 code = encode8(v, byte);
    if (live && c < cols16) gst<u2>(q.codes + row * q.ld + c, code);
    if (live && (threadIdx.x & 15) == 0) gst<uint8_t>(q.scales + (c / kCodeBlock) * q.lds + row, (uint8_t)byte);
}

constexpr int kGateRows = 16;      // rows of a workgroup's tile of 128 columns

template <int DT, int ACT>
__global__ __launch_bounds__(256) void gated_act_kernel(GateArgs a)
{
    const int64_t tc = (a.cols + 127) / 128, tiles = tc * ((a.rows + kGateRows - 1) / kGateRows);
    const int64_t cols16 = (a.cols + 15) & ~(int64_t)15;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t row = (t / tc) * kGateRows + threadIdx.x / 16, c = (t % tc) * 128 + 8 * (threadIdx.x & 15);
        const bool live = row < a.rows;
        const int cnt = live ? left8(c, a.cols) : 0;
        float g[8], u[8], y[8];
        load8<DT>(a.gate, row * a.ldg + c, cnt, g);
        load8<DT>(a.up, row * a.ldu + c, cnt, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = act<ACT, DT == kP32>(g[i]) * u[i];
        if (a.y) store8<DT>(a.y, row * a.ldy + c, cnt, y);
        if (a.q.codes) put_block(a.q, row, c, live, cols16, y);
        if (a.gq.codes) put_block(a.gq, row, c, live, cols16, g);
        if (a.uq.codes) put_block(a.uq, row, c, live, cols16, u);
    }
}

// ---- tiles of 128 x 128 whose transpose is coded too -----------------------
// 512 threads: thread t holds the eight columns of group t % 16 in the four
// rows of group t / 16.

constexpr int kTileThreads = 512;

struct TileLds {
    uint32_t cmax[8][128];                                       // largest magnitude of a column in a wave's 16 rows
    __attribute__((aligned(16))) uint8_t tr[128 * 128];          // codes by column
};

// Where the codes of rows 4 g .. 4 g + 3 of a column sit: the 16-byte chunk
// g / 4 is moved by the column's group, so that lanes which write the same rows
// of columns eight apart fall into different banks.
__device__ __forceinline__ int quad_at(int col, int g) { return col * 128 + 16 * ((g >> 2) ^ (col >> 3 & 7)) + 4 * (g & 3); }

// Codes of the transpose of the tile at (r0, c0): column c of the tile is row
// c0 + c of the coded matrix, its 128 rows one block.  Every thread calls it.
__device__ __forceinline__ void put_transposed(TileLds &lds, const Codes &q, int64_t r0, int64_t c0, int64_t rows, int64_t cols,
                                               const float (&v)[4][8])
{
    const int cl = threadIdx.x & 15, rg = threadIdx.x >> 4, wave = threadIdx.x >> 6;
    uint32_t m[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        m[k] = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) m[k] = max(m[k], fbits(v[i][k]) & 0x7FFFFFFFu);
        m[k] = rows_max_u32(m[k]);
    }
    __syncthreads();               // what the last call left in the LDS is read
    if ((threadIdx.x & 63) < 16) {
        *(u4 *)&lds.cmax[wave][8 * cl] = (u4){m[0], m[1], m[2], m[3]};
        *(u4 *)&lds.cmax[wave][8 * cl + 4] = (u4){m[4], m[5], m[6], m[7]};
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        uint32_t top = lds.cmax[0][8 * cl + k];
#pragma unroll
        for (int w = 1; w < 8; ++w) top = max(top, lds.cmax[w][8 * cl + k]);
        const uint32_t byte = block_scale(top);
        const float inv = block_inverse(byte);
        const uint32_t code = byte == 255u ? 0u : encode4(v[0][k], v[1][k], v[2][k], v[3][k], inv);
        *(uint32_t *)(lds.tr + quad_at(8 * cl + k, rg)) = code;
        if (rg == k && c0 + 8 * cl + k < cols) gst<uint8_t>(q.scales + (r0 / 128) * q.lds + c0 + 8 * cl + k, (uint8_t)byte);
    }
    __syncthreads();
    const int64_t rows16 = (rows + 15) & ~(int64_t)15;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int col = (threadIdx.x >> 3) + 64 * i, g = threadIdx.x & 7;      // 16 codes of a column
        if (c0 + col < cols && r0 + 16 * g < rows16)
            gst<u4>(q.codes + (c0 + col) * q.ld + r0 + 16 * g, *(const u4 *)(lds.tr + quad_at(col, 4 * g)));
    }
}

// Eight columns of a row of a coded matrix (zeros where it has none; code rows
// are padded to 16 with zero codes).
__device__ __forceinline__ void load_coded(const Codes &q, int64_t row, int64_t c, bool there, float v[8])
{
    u2 code = {0u, 0u};
    uint32_t byte = 127u;
    if (there) {
        code = gld<u2>(q.codes + row * q.ld + c);
        byte = gld<uint8_t>(q.scales + (c / kCodeBlock) * q.lds + row);
    }
    decode8(code, block_value(byte), v);
}

template <int DT, int ACT, bool CODED>
__global__ __launch_bounds__(kTileThreads) void gated_act_grad_kernel(GateGradArgs a)
{
    __shared__ TileLds lds;
    constexpr bool kFine = DT == kP32;
    const int cl = threadIdx.x & 15, rg = threadIdx.x >> 4;
    const int64_t tc = (a.cols + 127) / 128, tiles = tc * ((a.rows + 127) / 128);
    const int64_t cols16 = (a.cols + 15) & ~(int64_t)15;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t r0 = (t / tc) * 128, c0 = (t % tc) * 128;
        const int64_t c = c0 + 8 * cl, r = r0 + 4 * rg;
        const int have = left8(c, a.cols);
        float dg[4][8], du[4][8], y[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t row = r + i;
            const bool live = row < a.rows;
            const int cnt = live ? have : 0;
            float g[8], u[8], d[8];
            load8<DT>(a.dy, row * a.lddy + c, cnt, d);
            if (CODED) {
                load_coded(a.gq, row, c, cnt > 0, g);
                load_coded(a.uq, row, c, cnt > 0, u);
            } else {
                load8<DT>(a.gate, row * a.ldg + c, cnt, g);
                load8<DT>(a.up, row * a.ldu + c, cnt, u);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float s, slope;
                act_slope<ACT, kFine>(g[k], s, slope);
                // columns past the last one: a scale of infinity or NaN would make NaNs of their zero codes
                const bool in = k < cnt;
                dg[i][k] = in ? d[k] * u[k] * slope : 0.0f;
                du[i][k] = in ? d[k] * s : 0.0f;
                y[i][k] = in ? s * u[k] : 0.0f;
            }
            if (a.dgate) store8<DT>(a.dgate, row * a.lddg + c, cnt, dg[i]);
            if (a.dup) store8<DT>(a.dup, row * a.lddu + c, cnt, du[i]);
            if (a.dgq.codes) put_block(a.dgq, row, c, live, cols16, dg[i]);
            if (a.duq.codes) put_block(a.duq, row, c, live, cols16, du[i]);
        }
        if (a.dgt.codes) put_transposed(lds, a.dgt, r0, c0, a.rows, a.cols, dg);
        if (a.dut.codes) put_transposed(lds, a.dut, r0, c0, a.rows, a.cols, du);
        if (a.yt.codes) put_transposed(lds, a.yt, r0, c0, a.rows, a.cols, y);
    }
}

// Values of a coded matrix, and codes of its transpose.
template <int DT>
__global__ __launch_bounds__(kTileThreads) void block_restore_kernel(RestoreArgs a)
{
    __shared__ TileLds lds;
    const int cl = threadIdx.x & 15, rg = threadIdx.x >> 4;
    const int64_t tc = (a.cols + 127) / 128, tiles = tc * ((a.rows + 127) / 128);
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t r0 = (t / tc) * 128, c0 = (t % tc) * 128;
        const int64_t c = c0 + 8 * cl, r = r0 + 4 * rg;
        const int have = left8(c, a.cols);
        float v[4][8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int cnt = r + i < a.rows ? have : 0;
            load_coded(a.q, r + i, c, cnt > 0, v[i]);
#pragma unroll
            for (int k = 0; k < 8; ++k) v[i][k] = k < cnt ? v[i][k] : 0.0f;
            if (a.x) store8<DT>(a.x, (r + i) * a.ldx + c, cnt, v[i]);
        }
        if (a.qt.codes) put_transposed(lds, a.qt, r0, c0, a.rows, a.cols, v);
    }
}

// ---- launches --------------------------------------------------------------

static unsigned grid_of(int64_t tiles) { return (unsigned)(tiles < (1 << 20) ? tiles : 1 << 20); }

template <int DT, int ACT>
static hipError_t launch_gate_t(const GateArgs &a, hipStream_t st)
{
    const int64_t tiles = ((a.cols + 127) / 128) * ((a.rows + kGateRows - 1) / kGateRows);
    hipLaunchKernelGGL((gated_act_kernel<DT, ACT>), dim3(grid_of(tiles)), dim3(256), 0, st, a);
    return hipGetLastError();
}

template <int DT, int ACT>
static hipError_t launch_gate_grad_t(const GateGradArgs &a, hipStream_t st)
{
    const unsigned grid = grid_of(((a.cols + 127) / 128) * ((a.rows + 127) / 128));
    if (a.gate) hipLaunchKernelGGL((gated_act_grad_kernel<DT, ACT, false>), dim3(grid), dim3(kTileThreads), 0, st, a);
    else hipLaunchKernelGGL((gated_act_grad_kernel<DT, ACT, true>), dim3(grid), dim3(kTileThreads), 0, st, a);
    return hipGetLastError();
}

template <int DT>
static hipError_t launch_restore_t(const RestoreArgs &a, hipStream_t st)
{
    const unsigned grid = grid_of(((a.cols + 127) / 128) * ((a.rows + 127) / 128));
    hipLaunchKernelGGL((block_restore_kernel<DT>), dim3(grid), dim3(kTileThreads), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_gated_act(int dt, int act, const GateArgs &a, hipStream_t st)
{
    if (dt == kP32) return act == kActSilu ? launch_gate_t<kP32, kActSilu>(a, st) : launch_gate_t<kP32, kActGelu>(a, st);
    if (dt == kPBF16) return act == kActSilu ? launch_gate_t<kPBF16, kActSilu>(a, st) : launch_gate_t<kPBF16, kActGelu>(a, st);
    return act == kActSilu ? launch_gate_t<kPF16, kActSilu>(a, st) : launch_gate_t<kPF16, kActGelu>(a, st);
}

hipError_t launch_gated_act_grad(int dt, int act, const GateGradArgs &a, hipStream_t st)
{
    if (dt == kP32) return act == kActSilu ? launch_gate_grad_t<kP32, kActSilu>(a, st) : launch_gate_grad_t<kP32, kActGelu>(a, st);
    if (dt == kPBF16) return act == kActSilu ? launch_gate_grad_t<kPBF16, kActSilu>(a, st) : launch_gate_grad_t<kPBF16, kActGelu>(a, st);
    return act == kActSilu ? launch_gate_grad_t<kPF16, kActSilu>(a, st) : launch_gate_grad_t<kPF16, kActGelu>(a, st);
}

hipError_t launch_block_restore(int dt, const RestoreArgs &a, hipStream_t st)
{
    if (dt == kP32) return launch_restore_t<kP32>(a, st);
    if (dt == kPBF16) return launch_restore_t<kPBF16>(a, st);
    return launch_restore_t<kPF16>(a, st);
}

}  // namespace optstep
