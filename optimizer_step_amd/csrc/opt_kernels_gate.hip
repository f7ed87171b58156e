// opt_kernels_gate.hip -- the gated activation y = s(gate) * up with its
// inputs kept as block-coded 8-bit checkpoints, its backward pass from those
// codes or from the matrices, and the restoring of a coded matrix.
//
// s(x) = x sigma(p(x)), sigma the logistic function: p(x) = x is SiLU, p(x) =
// 2 sqrt(2/pi) (x + 0.044715 x^3) the tanh form of GELU (0.5 (1 + tanh(z)) =
// sigma(2 z)).  s'(x) = sigma (1 + x (1 - sigma) p'(x)).
//
// Bound by HBM where rows are whole eights.  8192 x 11008 bf16, SiLU: forward to
// codes with both inputs' codes 106 us (634 MB, 6.0 TB/s; the vector units are busy
// 70 % of the time); backward from those codes to both gradients' codes in both
// layouts and y's transposed 173 us (818 MB, 4.7 TB/s; a plain stream of four bytes
// in and five out takes 141).  2047 x 4096 fp16 from and to matrices 14.9 us; 8192 x
// 4096 codes restored as the transpose's 11.9 us (68 MB).  Sides that are no
// multiples, 8191 x 11005 bf16: from codes 177 us; GELU from matrices 231 (995 MB,
// 4.3 TB/s).  fp32, 8192 x 4096: from codes 82 us (4.5 TB/s), from matrices 141 (4.0).
#include "opt_pass.h"

namespace optstep {

// sigma(p) = sig * scale and rest = 1 - sigma(p).  FINE (32-bit results): each to a
// few binary32 units of itself.  Both come from e = exp(-|p|) <= 1, so nothing
// overflows or cancels, and what the rounding of |p| log2(e) costs, |p| 2^-24 of
// e, is put back (SiLU's |p| is held at 256, where e is 0, so that it is finite;
// GELU's is).  The hardware's exp2 gives 0 below 2^-126, where x e may still be a
// normal number: below p = -64, where 1 + e is 1 either way, e is formed 2^24
// times as large, and what sig makes is scaled back.
// 16-bit and 8-bit results do not see those: there exp(-p) may reach infinity, the
// exponent keeps the rounding of p log2(e), and sigma is 0 below 2^-126 (rest too,
// where it is multiplied by such a sigma).  To put the rounding back there took 112
// us for 107 (8192 x 11008, forward) and left as many of the gradients' codes off the
// exact ones as before.
// A NaN p may give any values: its x makes them NaN.
template <int ACT, bool FINE>
__device__ __forceinline__ void logistic(float p, float &sig, float &rest, float &scale)
{
    if (!FINE) {
        const float e = __builtin_amdgcn_exp2f(p * -1.44269504f);
        sig = __builtin_amdgcn_rcpf(1.0f + e);
        rest = __builtin_fminf(e, 0x1.fffffep127f) * sig;
        scale = 1.0f;
        return;
    }
    const float a = ACT == kActSilu ? __builtin_fminf(__builtin_fabsf(p), 256.0f) : __builtin_fabsf(p);
    const float t = a * -1.44269504f;
    const bool far = p < -64.0f;
    float e = __builtin_amdgcn_exp2f(t + (far ? 24.0f : 0.0f));        // (the sum is exact)
    // -a = t ln(2) + what t lacks
    const float lack = __builtin_fmaf(t, 1.90465438e-9f, __builtin_fmaf(t, -0.693147182f, -a));
    e = __builtin_fmaf(e, lack, e);
    const float big = __builtin_amdgcn_rcpf(1.0f + e), small = e * big;
    sig = p >= 0.0f ? big : small;
    rest = p >= 0.0f ? small : big;
    scale = far ? 0x1p-24f : 1.0f;
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
    float p, dp, sig, rest, scale;
    inner<ACT>(x, p, dp);
    logistic<ACT, FINE>(p, sig, rest, scale);
    return (x * sig) * scale;
}

template <int ACT, bool FINE>
__device__ __forceinline__ void act_slope(float x, float &s, float &slope)
{
    float p, dp, sig, rest, scale;
    inner<ACT>(x, p, dp);
    logistic<ACT, FINE>(p, sig, rest, scale);
    s = x * sig;
    slope = (ACT == kActSilu ? __builtin_fmaf(s, rest, sig) : __builtin_fmaf(s * rest, dp, sig)) * scale;
    s *= scale;
}

// One row's block of 128 columns by 16 lanes: codes and the scale's byte.
__device__ __forceinline__ void put_block(const Codes &q, int64_t row, int64_t c, bool live, int64_t cols16, const float v[8])
{
    uint32_t word;
    const u2 code = code_block(v, row16_max_u32(top8(v)), word);
    if (live && c < cols16) sst<u2>(q.codes + row * q.ld + c, code);
    if (live && (threadIdx.x & 15) == 0) gst<uint8_t>(q.scales + (c / kCodeBlock) * q.lds + row, (uint8_t)(word >> 23));
}

// Rows of a workgroup's tile of 128 columns: 16 lanes a row, one row each, so that
// many small waves keep the loads in flight.  Code stores carry the non-temporal
// hint (110 -> 106 us of the forward pass above); on the loads it costs 6 %, on
// results in 32 bits whose rows are not aligned 12 %.
constexpr int kGateRows = 16;

template <int DT, int ACT, bool EIGHTS>
__global__ __launch_bounds__(256) void gated_act_kernel(GateArgs a)
{
    const int64_t tc = (a.cols + 127) / 128, tiles = tc * ((a.rows + kGateRows - 1) / kGateRows);
    const int64_t cols16 = (a.cols + 15) & ~(int64_t)15;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t row = (t / tc) * kGateRows + threadIdx.x / 16, c = (t % tc) * 128 + 8 * (threadIdx.x & 15);
        const bool live = row < a.rows;
        const int cnt = live ? left8(c, a.cols) : 0;
        float g[8], u[8], y[8];
        load8<DT, EIGHTS>(a.gate, row * a.ldg + c, cnt, g);
        load8<DT, EIGHTS>(a.up, row * a.ldu + c, cnt, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = act<ACT, DT == kP32>(g[i]) * u[i];
        if (a.y) store8<DT, EIGHTS>(a.y, row * a.ldy + c, cnt, y);
        const Codes *const q[3] = {&a.q, &a.gq, &a.uq};
        const float *const v[3] = {y, g, u};
#pragma unroll
        for (int j = 0; j < 3; ++j) {
            if (q[j]->codes) put_block(*q[j], row, c, live, cols16, v[j]);
        }
    }
}

// The backward pass where no transpose is coded: dgate, dup and their codes, by
// rows.
template <int DT, int ACT, bool CODED, bool EIGHTS>
__global__ __launch_bounds__(256) void gated_act_grad_rows_kernel(GateGradArgs a)
{
    const int64_t tc = (a.cols + 127) / 128, tiles = tc * ((a.rows + kGateRows - 1) / kGateRows);
    const int64_t cols16 = (a.cols + 15) & ~(int64_t)15;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t row = (t / tc) * kGateRows + threadIdx.x / 16, c = (t % tc) * 128 + 8 * (threadIdx.x & 15);
        const bool live = row < a.rows;
        const int cnt = live ? left8(c, a.cols) : 0;
        float g[8], u[8], d[8], v[2][8];
        load8<DT, EIGHTS>(a.dy, row * a.lddy + c, cnt, d);
        if (CODED) {
            const Codes *const in[2] = {&a.gq, &a.uq};
            float *const out[2] = {g, u};
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                u2 code = {0u, 0u};
                uint32_t byte = 0;
                if (cnt > 0) {
                    code = gld<u2>(in[n]->codes + row * in[n]->ld + c);
                    byte = gld<uint8_t>(in[n]->scales + (c / kCodeBlock) * in[n]->lds + row);
                }
                decode8(code, byte, out[n]);
            }
        } else {
            load8<DT, EIGHTS>(a.gate, row * a.ldg + c, cnt, g);
            load8<DT, EIGHTS>(a.up, row * a.ldu + c, cnt, u);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            float s, slope;
            act_slope<ACT, DT == kP32>(g[k], s, slope);
            v[0][k] = d[k] * u[k] * slope;
            v[1][k] = d[k] * s;
            // columns past the last: a scale that says NaN makes NaNs of their zero codes
            if (CODED && !EIGHTS && k >= cnt) v[0][k] = v[1][k] = 0.0f;
        }
        if (a.dgate) store8<DT, EIGHTS>(a.dgate, row * a.lddg + c, cnt, v[0]);
        if (a.dup) store8<DT, EIGHTS>(a.dup, row * a.lddu + c, cnt, v[1]);
        const Codes *const q[2] = {&a.dgq, &a.duq};
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            if (q[n]->codes) put_block(*q[n], row, c, live, cols16, v[n]);
        }
    }
}

// ---- tiles of 128 x 128 whose transpose is coded too -----------------------
// 512 threads: thread t holds the eight columns of group t % 16 in the four
// rows of group t / 16.  The backward pass forms dgate first, then dup and y
// together from the inputs again, which stay as they are stored: 16-bit types in
// 128 registers, two workgroups a compute unit (GELU from matrices with sides that
// are no multiples of 128 spills one or two).  Whole tiles of bf16 from codes beside
// 165 to 169 us in the same runs: all
// three held at once (250 registers, one workgroup) 230, or in 128 registers 642
// (spills); s(gate) kept from part to part for two rows 175 (spills); every thread
// forming its columns' scales, one barrier less a part, 171; a persistent grid
// 181, with the next tile's loads ahead 215 (spills); tiles down the columns
// first 200.

constexpr int kTileThreads = 512;

// What a kernel knows of its matrix.  kFull: sides that are multiples of 128,
// so that every tile is whole.  kEights: columns a multiple of eight.
enum { kAnyShape = 0, kEights = 1, kFull = 2 };

// Where a thread's four rows of a tile begin: the address of the wave's first
// row is scalar work, a lane adds its group's distance from it.
struct Spot {
    char *p;
    int64_t step;          // bytes from a row to the next
    __device__ __forceinline__ char *row(int i) const { return p + i * step; }
};

template <int SIZE>
__device__ __forceinline__ Spot spot(const void *base, int64_t ld, int64_t r0, int64_t c0)
{
    const int64_t step = ld * SIZE;
    char *p = (char *)base + (r0 + 16 * wave_id()) * step + c0 * SIZE;
    return Spot{p + (int64_t)(threadIdx.x >> 4 & 3) * (4 * step) + (threadIdx.x & 15) * (8 * SIZE), step};
}

// How many of a thread's four rows exist, and of its eight columns (of a whole tile: all).
template <int SHAPE>
__device__ __forceinline__ int rows_of(int64_t rows, int64_t r0)
{
    if (SHAPE == kFull) return 4;
    const int left = (int)(rows - r0 < 128 ? rows - r0 : 128) - 4 * (int)(threadIdx.x >> 4);
    return left < 0 ? 0 : left > 4 ? 4 : left;
}

template <int SHAPE>
__device__ __forceinline__ int cols_of(int64_t cols, int64_t c0)
{
    if (SHAPE == kFull) return 8;
    const int left = (int)(cols - c0 < 128 ? cols - c0 : 128) - 8 * (int)(threadIdx.x & 15);
    return left < 0 ? 0 : left > 8 ? 8 : left;
}

template <int N>
struct TileLds {
    uint32_t top[N][128];                                        // bits of a column's largest magnitude, then its scale's word
    uint32_t lost;                                               // a column holds a NaN or an infinity
    __attribute__((aligned(16))) uint8_t tr[N][128 * 128];       // codes by column
};

// Where the codes of rows 4 g .. 4 g + 3 of a column sit: the 16-byte chunk
// g / 4 is moved by the column's group, so that lanes which write the same rows
// of columns eight apart fall into different banks.
__device__ __forceinline__ int quad_at(int col, int g) { return col * 128 + 16 * ((g >> 2) ^ (col >> 3 & 7)) + 4 * (g & 3); }

// Before any thread's add_tops, with a barrier between.
template <int N>
__device__ __forceinline__ void clear_tops(TileLds<N> &lds)
{
    if (threadIdx.x < N * 128) lds.top[0][threadIdx.x] = 0;
    if (threadIdx.x == 0) lds.lost = 0;
}

// Largest over the four rows of a wave of four columns' values, one column a
// row: each swap brings two columns together, each maximum halves their rows.
__device__ __forceinline__ uint32_t four_columns(const uint32_t m[4])
{
    const auto a = __builtin_amdgcn_permlane16_swap(m[0], m[1], false, false);
    const auto b = __builtin_amdgcn_permlane16_swap(m[2], m[3], false, false);
    const auto c = __builtin_amdgcn_permlane32_swap(max(a[0], a[1]), max(b[0], b[1]), false, false);
    return max(c[0], c[1]);
}

// A thread's largest magnitudes of its eight columns join the tile's.
__device__ __forceinline__ void add_tops(uint32_t (&top)[128], const float (&v)[4][8])
{
    uint32_t b[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) b[k] = fbits(__builtin_elementwise_maximum(max_abs(v[0][k], v[1][k]), max_abs(v[2][k], v[3][k])));
    uint32_t *const at = top + 8 * (threadIdx.x & 15) + (threadIdx.x >> 4 & 3);
    atomicMax(at, four_columns(b));
    atomicMax(at + 4, four_columns(b + 4));
}

// Between two barriers: the scales of the tile's columns, to the LDS and to the
// coded transpose; 128 threads, so that the others' columns cost them nothing.
template <int N>
__device__ __forceinline__ void set_scales(TileLds<N> &lds, int n, const Codes &q, int64_t r0, int64_t c0, int64_t cols)
{
    if (threadIdx.x >= 128) return;
    const uint32_t byte = block_scale(lds.top[n][threadIdx.x]);
    lds.top[n][threadIdx.x] = byte << 23;
    if (byte == 255u) lds.lost = 1;
    if (c0 + threadIdx.x < cols) gst<uint8_t>(q.scales + (r0 / 128) * q.lds + c0 + threadIdx.x, (uint8_t)byte);
}

// The tile's codes to the LDS, by column (a lost column's are put right on the
// way out).
template <int N>
__device__ __forceinline__ void code_columns(TileLds<N> &lds, int n, const float (&v)[4][8])
{
    const int cl = threadIdx.x & 15;
    const u4 x0 = *(const u4 *)(lds.top[n] + 8 * cl), x1 = *(const u4 *)(lds.top[n] + 8 * cl + 4);
#pragma unroll
    for (int k = 0; k < 8; ++k)
        *(uint32_t *)(lds.tr[n] + quad_at(8 * cl + k, threadIdx.x >> 4)) = codes4(v[0][k], v[1][k], v[2][k], v[3][k], k < 4 ? x0[k & 3] : x1[k & 3]);
}

// The coded transpose of a tile goes out of the LDS.
template <int SHAPE, int N>
__device__ __forceinline__ void put_tile(const TileLds<N> &lds, int n, const Codes &q, int64_t r0, int64_t c0, int64_t rows, int64_t cols)
{
    const int cols_left = (int)(cols - c0 < 128 ? cols - c0 : 128), rows_left = (int)(rows - r0 < 128 ? rows - r0 : 128);
    const int col = threadIdx.x >> 3, g = threadIdx.x & 7;      // 16 codes of a column
    char *const at = (char *)q.codes + (c0 + 8 * wave_id()) * q.ld + r0 + (int64_t)(col & 7) * q.ld + 16 * g;
    const bool lost = lds.lost != 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        u4 code = *(const u4 *)(lds.tr[n] + quad_at(col + 64 * i, 4 * g));
        if (lost && lds.top[n][col + 64 * i] == kLostWord) code = (u4){0u, 0u, 0u, 0u};
        if (SHAPE == kFull || (col + 64 * i < cols_left && 16 * g < rows_left)) gst<u4>(at + 64 * i * q.ld, code);
    }
}

// A thread's eight columns in its four rows of a coded matrix's tile, as they
// are stored (zeros where it has none; code rows are padded to 16 with zero
// codes, a block's scales to 4 rows).
struct CodedRows { u2 code[4]; uint32_t bytes; };

__device__ __forceinline__ CodedRows load_coded(const Codes &q, int64_t r0, int64_t c0, int live)
{
    const Spot at = spot<1>(q.codes, q.ld, r0, c0);
    CodedRows x;
    x.bytes = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x.code[i] = (u2){0u, 0u};
        if (i < live) x.code[i] = gld<u2>(at.row(i));
    }
    if (live > 0) x.bytes = gld<uint32_t>(q.scales + (c0 / kCodeBlock) * q.lds + r0 + 4 * (threadIdx.x >> 4));
    if (live < 4) x.bytes &= (1u << (8 * live)) - 1u;      // what stands past the last row is nobody's
    return x;
}

// Half of a thread's eight columns: four values.
__device__ __forceinline__ void half_of(const CodedRows &q, int i, int h, float v[4])
{
    const float x = bitsf((q.bytes >> (8 * i) & 255u) << 23);
    const f2_t lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q.code[i][h], x, false);
    const f2_t hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(q.code[i][h], x, true);
    v[0] = lo[0];
    v[1] = lo[1];
    v[2] = hi[0];
    v[3] = hi[1];
}

template <int DT>
struct RawRows { Raw<DT> row[4]; };

template <int DT>
__device__ __forceinline__ void half_of(const RawRows<DT> &q, int i, int h, float v[4])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (DT == kP32) {
            v[j] = bitsf(q.row[i].v[h & (DT == kP32)][j]);
        } else {
            const uint32_t w = q.row[i].v[0][2 * h + (j >> 1)];
            v[j] = DT == kPBF16 ? (j & 1 ? bf16_hi(w) : bf16_lo(w)) : (j & 1 ? f16_hi(w) : f16_lo(w));
        }
    }
}

template <int DT, int SHAPE>
__device__ __forceinline__ RawRows<DT> load_rows(const void *p, int64_t ld, int64_t r0, int64_t c0, int live, int have)
{
    const Spot at = spot<sizeof(typename Elem<DT>::T)>(p, ld, r0, c0);
    RawRows<DT> x;
#pragma unroll
    for (int i = 0; i < 4; ++i) x.row[i] = load_raw<DT, SHAPE != kAnyShape>(at.row(i), 0, i < live ? have : 0);
    return x;
}

// Forgets what was computed from these registers.
__device__ __forceinline__ void hold(CodedRows &q)
{
    asm volatile("" : "+v"(q.code[0]), "+v"(q.code[1]), "+v"(q.code[2]), "+v"(q.code[3]), "+v"(q.bytes));
}

template <int DT>
__device__ __forceinline__ void hold(RawRows<DT> &q)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        asm volatile("" : "+v"(q.row[i].v[0]));
        if (DT == kP32) asm volatile("" : "+v"(q.row[i].v[DT == kP32]));
    }
}

template <bool CODED, int DT> struct GateIn { typedef CodedRows T; };
template <int DT> struct GateIn<false, DT> { typedef RawRows<DT> T; };

// Four columns of row i: dgate (PART 0) to v[0], or dup and y (PART 1) to v[0]
// and v[1].  Columns past the last are zeros (a scale that says NaN makes NaNs of
// their zero codes).
template <int DT, int ACT, bool CODED, int SHAPE, int PART, class In>
__device__ __forceinline__ void grad4(const In &g, const In &u, const RawRows<DT> &d, int i, int h, int cnt, float (&v)[PART + 1][4][8])
{
    float gv[4], uv[4], dv[4];
    half_of(g, i, h, gv);
    half_of(u, i, h, uv);
    half_of(d, i, h, dv);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float s, slope;
        act_slope<ACT, DT == kP32>(gv[k], s, slope);
        v[0][i][4 * h + k] = PART == 0 ? dv[k] * uv[k] * slope : dv[k] * s;
        v[PART][i][4 * h + k] = PART == 0 ? v[0][i][4 * h + k] : s * uv[k];
        if (CODED && SHAPE == kAnyShape && 4 * h + k >= cnt) v[0][i][4 * h + k] = v[PART][i][4 * h + k] = 0.0f;
    }
}

// dgate or dup of a tile: as a matrix, and its codes by rows.
template <int DT, int SHAPE>
__device__ __forceinline__ void put_rows(const float (&v)[4][8], void *m, int64_t ld, const Codes &q, int64_t r0, int64_t c0, int64_t rows, int64_t cols)
{
    const int have = cols_of<SHAPE>(cols, c0), live = rows_of<SHAPE>(rows, r0);
    if (m) {
        const Spot at = spot<sizeof(typename Elem<DT>::T)>(m, ld, r0, c0);
#pragma unroll
        for (int i = 0; i < 4; ++i) store8<DT, SHAPE != kAnyShape>(at.row(i), 0, i < live ? have : 0, v[i]);
    }
    if (q.codes) {
        const Spot at = spot<1>(q.codes, q.ld, r0, c0);
        const bool padded = cols_of<SHAPE>((cols + 15) & ~(int64_t)15, c0) > 0;
        uint32_t mine = 0;             // lane i of a row keeps row i's scale: one store for the four
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t word;
            const u2 code = code_block(v[i], row16_max_u32(top8(v[i])), word);
            if (i < live && padded) gst<u2>(at.row(i), code);
            if ((threadIdx.x & 15) == i) mine = word;
        }
        if ((int)(threadIdx.x & 15) < live)
            gst<uint8_t>(q.scales + (c0 / kCodeBlock) * q.lds + r0 + 4 * (threadIdx.x >> 4) + (threadIdx.x & 15), (uint8_t)(mine >> 23));
    }
}

// The outputs of dgate, or of dup and y.
template <int DT, int ACT, bool CODED, int SHAPE, int PART, class In>
__device__ __forceinline__ void grad_part(const OPT_CONST GateGradArgs *a, TileLds<3> &lds, In &g, In &u, RawRows<DT> &d, int64_t r0, int64_t c0)
{
    a = again(a);
    hold(g);
    hold(u);
    hold(d);
    const int have = cols_of<SHAPE>(a->cols, c0), live = rows_of<SHAPE>(a->rows, r0);
    float v[PART + 1][4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) grad4<DT, ACT, CODED, SHAPE, PART>(g, u, d, i, h, i < live ? have : 0, v);
    const bool first = (PART ? a->dut.codes : a->dgt.codes) != nullptr, second = PART && a->yt.codes;
    if (first) add_tops(lds.top[PART], v[0]);
    if (second) add_tops(lds.top[2], v[PART]);
    if (PART) put_rows<DT, SHAPE>(v[0], a->dup, a->lddu, copy(a->duq), r0, c0, a->rows, a->cols);
    else put_rows<DT, SHAPE>(v[0], a->dgate, a->lddg, copy(a->dgq), r0, c0, a->rows, a->cols);
    __syncthreads();
    if (first) set_scales(lds, PART, PART ? copy(a->dut) : copy(a->dgt), r0, c0, a->cols);
    if (second) set_scales(lds, 2, copy(a->yt), r0, c0, a->cols);
    __syncthreads();
    if (first) code_columns(lds, PART, v[0]);
    if (second) code_columns(lds, 2, v[PART]);
}

template <int DT, int ACT, bool CODED, int SHAPE>
__device__ __forceinline__ void grad_tile(const OPT_CONST GateGradArgs *a, TileLds<3> &lds, int64_t r0, int64_t c0)
{
    const int have = cols_of<SHAPE>(a->cols, c0), live = rows_of<SHAPE>(a->rows, r0);
    typename GateIn<CODED, DT>::T g, u;
    if constexpr (CODED) {
        g = load_coded(copy(a->gq), r0, c0, have > 0 ? live : 0);
        u = load_coded(copy(a->uq), r0, c0, have > 0 ? live : 0);
    } else {
        g = load_rows<DT, SHAPE>(a->gate, a->ldg, r0, c0, live, have);
        u = load_rows<DT, SHAPE>(a->up, a->ldu, r0, c0, live, have);
    }
    RawRows<DT> d = load_rows<DT, SHAPE>(a->dy, a->lddy, r0, c0, live, have);
    clear_tops(lds);
    __syncthreads();
    // dgate first, then dup and y from the inputs again: the three at once would take 96 registers for the values alone
    grad_part<DT, ACT, CODED, SHAPE, 0>(a, lds, g, u, d, r0, c0);
    grad_part<DT, ACT, CODED, SHAPE, 1>(a, lds, g, u, d, r0, c0);
    __syncthreads();
    a = again(a);
    if (a->dgt.codes) put_tile<SHAPE>(lds, 0, copy(a->dgt), r0, c0, a->rows, a->cols);
    if (a->dut.codes) put_tile<SHAPE>(lds, 1, copy(a->dut), r0, c0, a->rows, a->cols);
    if (a->yt.codes) put_tile<SHAPE>(lds, 2, copy(a->yt), r0, c0, a->rows, a->cols);
}

// Waves a SIMD: four, in 128 registers, but two for 32-bit matrices (three operands
// of 32 registers a thread) and for 32-bit dy beside codes where columns are no
// multiple of eight (the code for single elements: 37 to 41 registers spilled in 128;
// 8191 x 4100 SiLU 175 us, 157 with two).  With whole eights four measure better
// though they spill 2 to 5 (8191 x 4104 from codes 111 us, 151 with two).
template <int DT, bool CODED, int SHAPE>
constexpr int grad_waves() { return DT == kP32 && (!CODED || SHAPE == kAnyShape) ? 2 : 4; }

template <int DT, int ACT, bool CODED, int SHAPE>
__global__ __launch_bounds__(kTileThreads, (grad_waves<DT, CODED, SHAPE>())) void gated_act_grad_kernel(GateGradArgs)
{
    __shared__ TileLds<3> lds;
    const OPT_CONST GateGradArgs *a = kernargs<GateGradArgs>();
    for (int64_t r0 = (int64_t)blockIdx.y * 128; r0 < a->rows; r0 += (int64_t)gridDim.y * 128)
        for (int64_t c0 = (int64_t)blockIdx.x * 128; c0 < a->cols; c0 += (int64_t)gridDim.x * 128) {
            if (r0 != (int64_t)blockIdx.y * 128 || c0 != (int64_t)blockIdx.x * 128) __syncthreads();    // the LDS of the last tile is read
            grad_tile<DT, ACT, CODED, SHAPE>(again(a), lds, r0, c0);
        }
}

// Values of a coded matrix, and codes of its transpose.
template <int DT, int SHAPE>
__device__ __forceinline__ void restore_tile(const OPT_CONST RestoreArgs *a, TileLds<1> &lds, int64_t r0, int64_t c0)
{
    const int have = cols_of<SHAPE>(a->cols, c0), live = rows_of<SHAPE>(a->rows, r0);
    const CodedRows q = load_coded(copy(a->q), r0, c0, have > 0 ? live : 0);
    const bool transposed = a->qt.codes;
    if (transposed) {
        clear_tops(lds);
        __syncthreads();
    }
    float v[4][8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        decode8(q.code[i], q.bytes >> (8 * i) & 255u, v[i]);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (SHAPE == kAnyShape && k >= (i < live ? have : 0)) v[i][k] = 0.0f;
    }
    if (a->x) {
        const Spot at = spot<sizeof(typename Elem<DT>::T)>(a->x, a->ldx, r0, c0);
#pragma unroll
        for (int i = 0; i < 4; ++i) store8<DT, SHAPE != kAnyShape>(at.row(i), 0, i < live ? have : 0, v[i]);
    }
    if (!transposed) return;
    add_tops(lds.top[0], v);
    __syncthreads();
    set_scales(lds, 0, copy(a->qt), r0, c0, a->cols);
    __syncthreads();
    code_columns(lds, 0, v);
    __syncthreads();
    put_tile<SHAPE>(lds, 0, copy(a->qt), r0, c0, a->rows, a->cols);
}

template <int DT, int SHAPE>
__global__ __launch_bounds__(kTileThreads) void block_restore_kernel(RestoreArgs)
{
    __shared__ TileLds<1> lds;
    const OPT_CONST RestoreArgs *a = kernargs<RestoreArgs>();
    for (int64_t r0 = (int64_t)blockIdx.y * 128; r0 < a->rows; r0 += (int64_t)gridDim.y * 128)
        for (int64_t c0 = (int64_t)blockIdx.x * 128; c0 < a->cols; c0 += (int64_t)gridDim.x * 128) {
            if (r0 != (int64_t)blockIdx.y * 128 || c0 != (int64_t)blockIdx.x * 128) __syncthreads();    // the LDS of the last tile is read
            restore_tile<DT, SHAPE>(again(a), lds, r0, c0);
        }
}

// ---- launches --------------------------------------------------------------

static unsigned grid_of(int64_t tiles) { return (unsigned)(tiles < (1 << 20) ? tiles : 1 << 20); }

// Tiles of 128 x 128: a workgroup each, of at most 2^20 (and 2^10 down).
static dim3 tiles_of(int64_t rows, int64_t cols)
{
    const int64_t x = (cols + 127) / 128, y = (rows + 127) / 128, most = (int64_t)1 << 20;
    const int64_t gy = y < 1024 ? y : 1024;
    return dim3((unsigned)(x < most / gy ? x : most / gy), (unsigned)gy);
}

template <int DT, int ACT>
static hipError_t launch_gate_t(const GateArgs &a, hipStream_t st)
{
    const int64_t tiles = ((a.cols + 127) / 128) * ((a.rows + kGateRows - 1) / kGateRows);
    if (a.cols % 8 == 0) hipLaunchKernelGGL((gated_act_kernel<DT, ACT, true>), dim3(grid_of(tiles)), dim3(256), 0, st, a);
    else hipLaunchKernelGGL((gated_act_kernel<DT, ACT, false>), dim3(grid_of(tiles)), dim3(256), 0, st, a);
    return hipGetLastError();
}

static int shape_of(int64_t rows, int64_t cols) { return rows % 128 == 0 && cols % 128 == 0 ? kFull : cols % 8 == 0 ? kEights : kAnyShape; }

template <int DT, int ACT, bool CODED>
static hipError_t launch_gate_grad_t(const GateGradArgs &a, hipStream_t st)
{
    if (!a.dgt.codes && !a.dut.codes && !a.yt.codes) {
        const unsigned grid = grid_of(((a.cols + 127) / 128) * ((a.rows + kGateRows - 1) / kGateRows));
        if (a.cols % 8 == 0) hipLaunchKernelGGL((gated_act_grad_rows_kernel<DT, ACT, CODED, true>), dim3(grid), dim3(256), 0, st, a);
        else hipLaunchKernelGGL((gated_act_grad_rows_kernel<DT, ACT, CODED, false>), dim3(grid), dim3(256), 0, st, a);
        return hipGetLastError();
    }
    const dim3 grid = tiles_of(a.rows, a.cols);
    switch (shape_of(a.rows, a.cols)) {
    case kFull: hipLaunchKernelGGL((gated_act_grad_kernel<DT, ACT, CODED, kFull>), grid, dim3(kTileThreads), 0, st, a); break;
    case kEights: hipLaunchKernelGGL((gated_act_grad_kernel<DT, ACT, CODED, kEights>), grid, dim3(kTileThreads), 0, st, a); break;
    default: hipLaunchKernelGGL((gated_act_grad_kernel<DT, ACT, CODED, kAnyShape>), grid, dim3(kTileThreads), 0, st, a);
    }
    return hipGetLastError();
}

template <int DT, int ACT>
static hipError_t launch_gate_grad_a(const GateGradArgs &a, hipStream_t st)
{
    return a.gate ? launch_gate_grad_t<DT, ACT, false>(a, st) : launch_gate_grad_t<DT, ACT, true>(a, st);
}

template <int DT>
static hipError_t launch_restore_t(const RestoreArgs &a, hipStream_t st)
{
    const dim3 grid = tiles_of(a.rows, a.cols);
    switch (shape_of(a.rows, a.cols)) {
    case kFull: hipLaunchKernelGGL((block_restore_kernel<DT, kFull>), grid, dim3(kTileThreads), 0, st, a); break;
    case kEights: hipLaunchKernelGGL((block_restore_kernel<DT, kEights>), grid, dim3(kTileThreads), 0, st, a); break;
    default: hipLaunchKernelGGL((block_restore_kernel<DT, kAnyShape>), grid, dim3(kTileThreads), 0, st, a);
    }
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
    if (dt == kP32) return act == kActSilu ? launch_gate_grad_a<kP32, kActSilu>(a, st) : launch_gate_grad_a<kP32, kActGelu>(a, st);
    if (dt == kPBF16) return act == kActSilu ? launch_gate_grad_a<kPBF16, kActSilu>(a, st) : launch_gate_grad_a<kPBF16, kActGelu>(a, st);
    return act == kActSilu ? launch_gate_grad_a<kPF16, kActSilu>(a, st) : launch_gate_grad_a<kPF16, kActGelu>(a, st);
}

hipError_t launch_block_restore(int dt, const RestoreArgs &a, hipStream_t st)
{
    if (dt == kP32) return launch_restore_t<kP32>(a, st);
    if (dt == kPBF16) return launch_restore_t<kPBF16>(a, st);
    return launch_restore_t<kPF16>(a, st);
}

}  // namespace optstep
