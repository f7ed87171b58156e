// opt_kernels_drop.hip -- dropout from the counter-based generator.
//
// out_j = res_j + (r_j >= T ? x_j * s : 0), with r_j the 16 bits of element j
// in its stream; the mask is recomputed wherever it is needed and never
// stored, so the backward pass is the same kernel on the gradient.
//
// Bound by HBM: 8192 x 4096 bf16 with a residual takes 32.3 us (201 MB, 6.2
// TB/s).  Sixteen bits an element keep the generator below that: one block of
// it, about 160 issue cycles, serves eight elements, and the vector units are
// busy 32 % of the time; p is then a multiple of 2^-16.  Loads and stores carry
// the non-temporal hint (37.6 us without).
#include "opt_pass.h"

namespace optstep {

constexpr int kDropThreads = 256;
// Groups of eight elements a lane takes: 32 bytes of either type (4.2 M fp32
// elements 8.0 us, with two groups 8.8; 33.6 M bf16 23.6, with one 25.5).
constexpr int drop_groups(int dt) { return dt == kP32 ? 1 : 2; }

// One Philox4x32-10 block serves eight elements, 16 bits each: element j takes
// half j%2 of word (j%8)/2 of the block with counter (j>>3 low, j>>35 | 2^31,
// offset low, offset high).  Bit 31 of the second word keeps the stream apart
// from the rounding cast's with the same seed and offset.
template <int DT, bool RES>
__global__ __launch_bounds__(kDropThreads) void dropout_kernel(DropArgs a)
{
    constexpr int kDropGroups = drop_groups(DT), kDropTile = kDropThreads * kDropGroups * 8;
    const int64_t ngroups = (a.n + 7) / 8;
    const int64_t ntiles = (a.n + kDropTile - 1) / kDropTile;
    for (int64_t t = blockIdx.x; t < ntiles; t += gridDim.x) {
        const int64_t g0 = t * (kDropTile / 8) + threadIdx.x;
        float x[kDropGroups][8], r[kDropGroups][8];
#pragma unroll
        for (int u = 0; u < kDropGroups; ++u) {
            const int64_t g = g0 + u * kDropThreads;
            const int cnt = left8(8 * g, a.n);
            load8<DT, false, true>(a.x, 8 * g, cnt, x[u]);
            if (RES) load8<DT, false, true>(a.res, 8 * g, cnt, r[u]);
        }
#pragma unroll
        for (int u = 0; u < kDropGroups; ++u) {
            const int64_t g = g0 + u * kDropThreads;
            if (g >= ngroups) break;
            const uint64_t q = (uint64_t)(a.base8 + g);
            const PhiloxOut o = philox4x32_10((uint32_t)q, (uint32_t)(q >> 32) | 0x80000000u, (uint32_t)a.offset,
                                              (uint32_t)(a.offset >> 32), (uint32_t)a.seed, (uint32_t)(a.seed >> 32));
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t w = philox_word(o, i >> 1);
                const uint32_t bits = i & 1 ? w >> 16 : w & 0xFFFFu;
                v[i] = bits >= a.threshold ? x[u][i] * a.scale : 0.0f;
                if (RES) v[i] = v[i] + r[u][i];
            }
            store8<DT, false, true>(a.out, 8 * g, left8(8 * g, a.n), v);
        }
    }
}

template <int DT>
static hipError_t launch_dropout_t(const DropArgs &a, hipStream_t st)
{
    constexpr int kDropTile = kDropThreads * drop_groups(DT) * 8;
    const int64_t tiles = (a.n + kDropTile - 1) / kDropTile;
    const unsigned grid = (unsigned)(tiles < (1 << 20) ? tiles : 1 << 20);
    if (a.res) hipLaunchKernelGGL((dropout_kernel<DT, true>), dim3(grid), dim3(kDropThreads), 0, st, a);
    else hipLaunchKernelGGL((dropout_kernel<DT, false>), dim3(grid), dim3(kDropThreads), 0, st, a);
    return hipGetLastError();
}

hipError_t launch_dropout(int dt, const DropArgs &a, hipStream_t st)
{
    if (dt == kP32) return launch_dropout_t<kP32>(a, st);
    if (dt == kPBF16) return launch_dropout_t<kPBF16>(a, st);
    return launch_dropout_t<kPF16>(a, st);
}

}  // namespace optstep
