// opt_kernels_cast.hip -- the cast to block-coded matrices: E4M3 codes with
// one power-of-two scale for each row (or each 128 rows) and 128 columns, of
// the matrix and/or of its transpose, in one read of it.
#include "opt_pass.h"

namespace optstep {

constexpr int kCastRow = 144;      // bytes of a column in the LDS transpose (128 codes, padded)

// One 128 x 128 tile a workgroup.  Thread t holds the eight columns of group
// t % 16 in the eight rows of group t / 16: a row's block maximum is one DPP
// row, a column's codes of eight rows are one 8-byte LDS store.
template <int DT, bool SQUARE>
__global__ __launch_bounds__(256) void block_cast_kernel(CastArgs a)
{
    __shared__ uint32_t cmax[4][128];
    __shared__ __attribute__((aligned(16))) uint8_t tr[128 * kCastRow];
    const int cl = threadIdx.x & 15, rg = threadIdx.x >> 4, wave = threadIdx.x >> 6;
    const int64_t tc = (a.cols + 127) / 128, tiles = tc * ((a.rows + 127) / 128);
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t r0 = (t / tc) * 128, c0 = (t % tc) * 128;
        const int64_t c = c0 + 8 * cl, r = r0 + 8 * rg;
        const int cnt = left8(c, a.cols);
        float v[8][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) load8<DT>(a.x, (r + i) * a.ldx + c, r + i < a.rows ? cnt : 0, v[i]);
        uint32_t rm[8], cm[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) cm[i] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            rm[i] = abs_max8(v[i]);
#pragma unroll
            for (int k = 0; k < 8; ++k) cm[k] = max(cm[k], fbits(v[i][k]) & 0x7FFFFFFFu);
        }
        __syncthreads();           // the LDS of the last tile is read
        if (SQUARE) {
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, rm[i]);
            m = wave_max_u32(m);
            if ((threadIdx.x & 63) == 0) cmax[wave][0] = m;
        } else if (a.qt.codes) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                uint32_t m = cm[k];
                m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
                m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
                if ((threadIdx.x & 63) < 16) cmax[wave][8 * cl + k] = m;
            }
        }
        __syncthreads();
        uint32_t square = 0;
        if (SQUARE) square = block_scale(max(max(cmax[0][0], cmax[1][0]), max(cmax[2][0], cmax[3][0])));
        if (a.q.codes) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t byte = SQUARE ? square : block_scale(row16_max_u32(rm[i]));
                const u2 code = encode8(v[i], byte);
                if (r + i < a.rows) {
                    if (c < ((a.cols + 15) & ~(int64_t)15)) gst<u2>(a.q.codes + (r + i) * a.q.ld + c, code);
                    if (cl == 0) gst<uint8_t>(a.q.scales + (c0 / 128) * a.q.lds + r + i, (uint8_t)byte);
                }
            }
        }
        if (a.qt.codes) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                uint32_t byte = square;
                if (!SQUARE) byte = block_scale(max(max(cmax[0][8 * cl + k], cmax[1][8 * cl + k]), max(cmax[2][8 * cl + k], cmax[3][8 * cl + k])));
                const float col[8] = {v[0][k], v[1][k], v[2][k], v[3][k], v[4][k], v[5][k], v[6][k], v[7][k]};
                *(u2 *)(tr + (8 * cl + k) * kCastRow + 8 * rg) = encode8(col, byte);
                if (rg == 0 && c + k < a.cols) gst<uint8_t>(a.qt.scales + (r0 / 128) * a.qt.lds + c + k, (uint8_t)byte);
            }
            __syncthreads();
            const int64_t rows16 = (a.rows + 15) & ~(int64_t)15;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int col = (threadIdx.x >> 3) + 32 * i, part = 16 * (threadIdx.x & 7);
                if (c0 + col < a.cols && r0 + part < rows16)
                    gst<u4>(a.qt.codes + (c0 + col) * a.qt.ld + r0 + part, *(const u4 *)(tr + col * kCastRow + part));
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
