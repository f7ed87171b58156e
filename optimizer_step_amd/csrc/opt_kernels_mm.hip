// opt_kernels_mm.hip -- the product of two block-coded matrices,
// C[m, n] = sum_k A[m, k] B[n, k] (+ C), on the matrix cores.
//
// The matrix cores' 8-bit products line up each sixteen of them by the largest
// one's exponent and keep 14 bits below it (found by probing single terms),
// which leaves a sum 1.5e-5 off on normal data; their BF16 products are exact
// and are summed in binary32 (1e-8 off).  An E4M3 code times its power-of-two
// scale is exact in BF16, and gfx950 converts two with their scale in one
// instruction: that is the form used here.
//
// B's rows go in as the instruction's first operand: a lane then ends with
// four neighbouring columns of C, which it stores together.
#include "opt_pass.h"

namespace optstep {

typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf2v __attribute__((ext_vector_type(2)));

// A scale byte as the binary32 number 2^(byte - 127) (whose exponent field is
// what the conversion takes: 255 gives NaNs).
__device__ __forceinline__ float scale_of(uint32_t byte) { return bitsf(byte ? byte << 23 : 0x00400000u); }

// Eight codes times their scale, exact (a product below 2^-126 may read as 0).
__device__ __forceinline__ bf8v widen8(uint32_t lo, uint32_t hi, float scale)
{
    const bf2v a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    const bf2v b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    const bf2v c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    const bf2v d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return (bf8v){a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// 32 code bytes of one row for a lane, widened.  Which 32 of the block's 128
// columns they are does not matter to the sum as long as A and B agree: a lane
// takes two 16-byte pieces 64 columns apart, so each quarter-wave reads 64
// consecutive bytes.  Pieces past the row's end read as zero codes.
struct Piece { bf8v v[4]; };

__device__ __forceinline__ Piece code_piece(const uint8_t *row, const uint8_t *scale, int64_t k0, int64_t k, int part)
{
    const u4 z = {0, 0, 0, 0};
    const int64_t p = k0 + 16 * part;
    const u4 lo = p < k ? gld<u4>(row + p) : z;
    const u4 hi = p + 64 < k ? gld<u4>(row + p + 64) : z;
    const float s = scale_of(gld<uint8_t>(scale));
    return Piece{{widen8(lo[0], lo[1], s), widen8(lo[2], lo[3], s), widen8(hi[0], hi[1], s), widen8(hi[2], hi[3], s)}};
}

template <int DT>
__device__ __forceinline__ void store_c(const MatmulArgs &a, int64_t m, int64_t n, f4 v)
{
    if (m >= a.m) return;
    typedef typename Elem<DT>::T T;
    T *p = (T *)a.c + m * a.ldc + n;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (n + i >= a.n) return;
        float x = v[i];
        float old[8];
        if (a.accumulate) {
            load8<DT>(p, i, 1, old);
            x = old[0] + x;
        }
        if (DT == kP32) gst<float>(p + i, x);
        else gst<uint16_t>(p + i, (uint16_t)pack2<DT>(x, 0.0f));
    }
}

// A workgroup of four waves forms 16 x MT rows of A by 16 of B; each wave sums
// every fourth block of 128 columns and the four sums meet in LDS.
template <int DT, int MT>
__global__ __launch_bounds__(256) void product_rows_kernel(MatmulArgs a)
{
    __shared__ f4 sum[3][MT][64];
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, r = lane & 15, part = lane >> 4;
    const int64_t tn = (a.n + 15) / 16, tiles = tn * ((a.m + 16 * MT - 1) / (16 * MT));
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t n0 = (t % tn) * 16, m0 = (t / tn) * (16 * MT);
        const int64_t nr = min(n0 + r, a.n - 1);
        int64_t mr[MT];
        f4 acc[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            mr[i] = min(m0 + 16 * i + r, a.m - 1);
            acc[i] = (f4){0, 0, 0, 0};
        }
        for (int64_t k0 = 128 * wave; k0 < a.k; k0 += 512) {
            const Piece b = code_piece(a.b.codes + nr * a.b.ld, a.b.scales + (k0 / 128) * a.b.lds + nr, k0, a.k, part);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const Piece x = code_piece(a.a.codes + mr[i] * a.a.ld, a.a.scales + (k0 / 128) * a.a.lds + mr[i], k0, a.k, part);
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b.v[j], x.v[j], acc[i], 0, 0, 0);
            }
        }
        __syncthreads();
        if (wave > 0)
#pragma unroll
            for (int i = 0; i < MT; ++i) sum[wave - 1][i][lane] = acc[i];
        __syncthreads();
        if (wave == 0)
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const f4 v = ((acc[i] + sum[0][i][lane]) + sum[1][i][lane]) + sum[2][i][lane];
                store_c<DT>(a, m0 + 16 * i + r, n0 + 4 * part, v);
            }
    }
}

template <int DT>
static hipError_t launch_matmul_t(const MatmulArgs &a, hipStream_t st)
{
    const int64_t tiles = ((a.n + 15) / 16) * ((a.m + 15) / 16);
    const unsigned grid = (unsigned)(tiles < (1 << 20) ? tiles : 1 << 20);
    hipLaunchKernelGGL((product_rows_kernel<DT, 1>), dim3(grid), dim3(256), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_block_matmul(int dt, const MatmulArgs &a, hipStream_t st)
{
    if (dt == kP32) return launch_matmul_t<kP32>(a, st);
    if (dt == kPBF16) return launch_matmul_t<kPBF16>(a, st);
    return launch_matmul_t<kPF16>(a, st);
}

}  // namespace optstep
