// opt_kernels_cast.hip -- the cast to block-coded matrices: E4M3 codes with
// one power-of-two scale X for each row (or each 128 rows) and 128 columns, of
// the matrix and/or of its transpose, in one read of it.
//
// X is the smallest power of two with A <= 448 X (A the block's largest
// magnitude): x / X is exact and never leaves the grid, so a code is one
// conversion.  The tile is 128 x 128 because the transpose's blocks are 128
// rows tall: both layouts' maxima and codes come from one read.  Bound by HBM
// on the way in and out: both layouts of 8192 x 4096 bf16 take 28.3 us (134 MB,
// 4.7 TB/s), one layout 20 to 22 us, a 11008 x 4096 fp32 weight 51.8 us (271 MB,
// 5.2 TB/s); the vector units are busy 41 and 21 % of the time.
#include "opt_pass.h"

namespace optstep {

// Largest of a lane's value and those 16 and 32 lanes away: of the four rows
// of a wave, in every lane.
__device__ __forceinline__ uint32_t rows_max_u32(uint32_t v)
{
    auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(p[0], p[1]);
    p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return max(p[0], p[1]);
}

// Where the codes of rows 8 g .. 8 g + 7 of a column sit in the transposed
// tile: 16 lanes that write the same rows of columns eight apart, and 8 that
// read one column's, each fall into different banks.
__device__ __forceinline__ int tr_at(int col, int g) { return col * 128 + 8 * (g ^ (col >> 3 & 15)); }

// Keeps the tile in its stored form: widened values are formed again where they
// are used, not held over (152 registers of a 16-bit type instead of 203: 31.6 -> 28.3 us at 8192 x 4096, both layouts).
template <int DT>
__device__ __forceinline__ void hold(Raw<DT> (&x)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        asm volatile("" : "+v"(x[i].v[0]));
        if (DT == kP32) asm volatile("" : "+v"(x[i].v[DT == kP32]));
    }
}

template <int DT>
__device__ __forceinline__ float raw_at(const Raw<DT> &r, int k)
{
    if (DT == kP32) return bitsf(r.v[k >> 2 & (DT == kP32)][k & 3]);
    const uint32_t w = r.v[0][k >> 1 & 3];
    if (DT == kPBF16) return k & 1 ? bf16_hi(w) : bf16_lo(w);
    return k & 1 ? f16_hi(w) : f16_lo(w);
}

// One 128 x 128 tile a workgroup.  Thread t holds the eight columns of group
// t % 16 in the eight rows of group t / 16: a row's block maximum is one DPP
// row, a column's codes of eight rows are one 8-byte LDS store.
template <int DT, bool SQUARE>
__global__ __launch_bounds__(256) void block_cast_kernel(CastArgs a)
{
    __shared__ uint32_t cmax[4][128];
    __shared__ __attribute__((aligned(16))) uint8_t tr[128 * 128];
    const int cl = threadIdx.x & 15, rg = threadIdx.x >> 4, wave = threadIdx.x >> 6;
    const int64_t tc = (a.cols + 127) / 128, tiles = tc * ((a.rows + 127) / 128);
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t r0 = (t / tc) * 128, c0 = (t % tc) * 128;
        const int64_t c = c0 + 8 * cl, r = r0 + 8 * rg;
        const int cnt = left8(c, a.cols), live = left8(r, a.rows);       // columns and rows that exist
        Raw<DT> x[8];
        // the matrix is read once: the non-temporal hint, 57 -> 53 us at 11008 x 4096 fp32
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = load_raw<DT, false, true>(a.x, (r + i) * a.ldx + c, i < live ? cnt : 0);
        uint32_t rm[8], cm[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) cm[k] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v[8];
            unpack_raw<DT>(x[i], v);
            rm[i] = abs_max8(v);
#pragma unroll
            for (int k = 0; k < 8; ++k) cm[k] = max(cm[k], fbits(v[k]) & 0x7FFFFFFFu);
        }
        hold<DT>(x);
        __syncthreads();           // the LDS of the last tile is read
        if (SQUARE) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, rm[i]);
            m = wave_max_u32(m);
            if ((threadIdx.x & 63) == 0) cmax[wave][0] = m;
        } else if (a.qt.codes) {
#pragma unroll
            for (int k = 0; k < 8; ++k) cm[k] = rows_max_u32(cm[k]);
            if ((threadIdx.x & 63) < 16) {
                *(u4 *)&cmax[wave][8 * cl] = (u4){cm[0], cm[1], cm[2], cm[3]};
                *(u4 *)&cmax[wave][8 * cl + 4] = (u4){cm[4], cm[5], cm[6], cm[7]};
            }
        }
        __syncthreads();
        uint32_t square = 0;
        if (SQUARE) square = block_scale(max(max(cmax[0][0], cmax[1][0]), max(cmax[2][0], cmax[3][0])));
        if (a.q.codes) {
            uint32_t mine = square;        // lane i of a row keeps row i's scale: one store for the eight
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t byte = SQUARE ? square : block_scale(row16_max_u32(rm[i]));
                if (!SQUARE && cl == i) mine = byte;
                float v[8];
                unpack_raw<DT>(x[i], v);
                const u2 code = encode8(v, byte);
                if (i < live && c < ((a.cols + 15) & ~(int64_t)15)) gst<u2>(a.q.codes + (r + i) * a.q.ld + c, code);
            }
            if (cl < live) gst<uint8_t>(a.q.scales + (c0 / 128) * a.q.lds + r + cl, (uint8_t)mine);
        }
        if (a.qt.codes) {
            hold<DT>(x);
            uint32_t byte[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) byte[k] = square;
            if (!SQUARE) {
#pragma unroll
                for (int k = 0; k < 8; k += 4) {
                    const u4 m0 = *(const u4 *)&cmax[0][8 * cl + k], m1 = *(const u4 *)&cmax[1][8 * cl + k];
                    const u4 m2 = *(const u4 *)&cmax[2][8 * cl + k], m3 = *(const u4 *)&cmax[3][8 * cl + k];
#pragma unroll
                    for (int i = 0; i < 4; ++i) byte[k + i] = block_scale(max(max(m0[i], m1[i]), max(m2[i], m3[i])));
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float col[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) col[i] = raw_at<DT>(x[i], k);
                *(u2 *)(tr + tr_at(8 * cl + k, rg)) = encode8(col, byte[k]);
            }
            uint32_t mine = byte[0];
#pragma unroll
            for (int k = 1; k < 8; ++k)
                if (rg == k) mine = byte[k];
            if (rg < cnt) gst<uint8_t>(a.qt.scales + (r0 / 128) * a.qt.lds + c + rg, (uint8_t)mine);
            __syncthreads();
            const int64_t rows16 = (a.rows + 15) & ~(int64_t)15;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int col = (threadIdx.x >> 3) + 32 * i, g = 2 * (threadIdx.x & 7);
                if (c0 + col < a.cols && r0 + 8 * g < rows16) {
                    const u2 lo = *(const u2 *)(tr + tr_at(col, g)), hi = *(const u2 *)(tr + tr_at(col, g + 1));
                    gst<u4>(a.qt.codes + (c0 + col) * a.qt.ld + r0 + 8 * g, (u4){lo[0], lo[1], hi[0], hi[1]});
                }
            }
        }
    }
}

template <int DT>
static hipError_t launch_cast_t(const CastArgs &a, int square, hipStream_t st)
{
    const int64_t tiles = ((a.cols + 127) / 128) * ((a.rows + 127) / 128);
    const unsigned grid = (unsigned)(tiles < (1 << 20) ? tiles : 1 << 20);
    if (square) hipLaunchKernelGGL((block_cast_kernel<DT, true>), dim3(grid), dim3(256), 0, st, a);
    else hipLaunchKernelGGL((block_cast_kernel<DT, false>), dim3(grid), dim3(256), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_block_cast(int dt, const CastArgs &a, int square, hipStream_t st)
{
    if (dt == kP32) return launch_cast_t<kP32>(a, square, st);
    if (dt == kPBF16) return launch_cast_t<kPBF16>(a, square, st);
    return launch_cast_t<kPF16>(a, square, st);
}

}  // namespace optstep
