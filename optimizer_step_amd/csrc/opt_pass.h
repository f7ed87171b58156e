// opt_pass.h -- what the training-pass operators beside the step share:
// dropout, the RMS norm, the cast to block-coded matrices, their product, the
// gated activation, the heads' norm and restored codes.  Kernel argument
// records, loads and stores of eight elements, sums over lanes, and the codecs of
// one 128-element block.
#pragma once

#include "opt_device.h"

namespace optstep {

constexpr int kCodeBlock = 128;    // columns that share one scale of a block-coded matrix
constexpr int64_t kMaxNormCols = 32768;   // longest row of the norms (a row stays in registers)

// A block-coded matrix (opt_codes in opt_step.h).
struct Codes {
    uint8_t *codes;
    int64_t ld;
    uint8_t *scales;
    int64_t lds;
};

struct DropArgs {
    const void *x, *res;
    void *out;
    int64_t n;
    int64_t base8;         // index_base / 8: block of element 0 in the stream
    uint64_t seed, offset;
    uint32_t threshold;    // an element is dropped if its 16 bits are below this
    float scale;
};

struct NormArgs {
    int64_t rows, cols;
    const void *x, *res, *w;
    void *h, *y;
    int64_t ldx, ldr, ldh, ldy;
    Codes q;
    int w_dtype;
    double eps, inv_cols;  // inv_cols: 1 / cols
};

struct NormGradArgs {
    int64_t rows, cols;
    const void *dy, *h, *w, *dh;
    void *dx;
    int64_t lddy, ldh, lddh, lddx;
    float *part;           // [groups][cols] partial sums of the weight's gradient, or null
    int w_dtype;
    double eps, inv_cols;  // inv_cols: 1 / cols
};

struct CastArgs {
    int64_t rows, cols, ldx;
    const void *x;
    Codes q, qt;           // codes null: that layout is not written
};

struct MatmulArgs {
    int64_t m, n, k;       // k: bytes of a code row, a multiple of 16
    Codes a, b;
    void *c;
    int64_t ldc;
    int accumulate;
    int exact;             // 0: a 16-bit c may take the 8-bit products
};

constexpr int kActSilu = 0, kActGelu = 1;
constexpr int kMaxHeadDim = 512;   // longest head (a head stays in a wave's registers)

struct GateArgs {
    int64_t rows, cols;
    const void *gate, *up;
    void *y;
    int64_t ldg, ldu, ldy;
    Codes q, gq, uq;       // codes null: not written
};

struct GateGradArgs {
    int64_t rows, cols;
    const void *dy, *gate, *up;    // gate null: from gq and uq
    void *dgate, *dup;
    int64_t lddy, ldg, ldu, lddg, lddu;
    Codes gq, uq;
    Codes dgq, duq, dgt, dut, yt;  // codes null: not written
};

struct RestoreArgs {
    int64_t rows, cols;
    Codes q;
    void *x;               // null: not written
    int64_t ldx;
    Codes qt;              // codes null: not written
};

// The queries or the keys of a call (strides in elements).
struct HeadSet {
    int64_t heads;
    const void *x, *w;
    void *y;
    int64_t xt, xh, yt, yh;
    Codes q;
};

struct HeadGradSet {
    int64_t heads;
    const void *dy, *x, *w;        // x null: from q
    void *dx;
    int64_t dyt, dyh, xt, xh, dxt, dxh;
    Codes q;
};

// What both passes of the heads share.
struct HeadTurn {
    int64_t tokens, table_rows, ldt;
    const float *table;
    const void *positions; // null: token t stands at row t
    int dim, rot;
    int wide_positions;    // 64-bit
    int neighbours;        // pairs (2 i, 2 i + 1), not (i, i + rot/2)
    int w_dtype;
    double eps, inv_dim;
};

struct HeadArgs {
    HeadTurn t;
    HeadSet s[2];
};

struct HeadGradArgs {
    HeadTurn t;
    HeadGradSet s[2];
    double *part;          // [groups][2][dim] partial sums of the weights' gradients, or null
};

// Workgroups of the heads' backward pass, by the tokens alone (so that the order
// of the weights' sums is too).
int64_t head_grad_groups(int64_t tokens);

// Lanes of a row and workgroups of the norm's backward pass, by the shape
// alone (so that the weight gradient's order of addition is too).
struct NormShape {
    int lanes;             // lanes that hold one row: 16, 64, 256 or 1024
    int vecs;              // groups of eight elements a lane holds
};
NormShape norm_shape(int64_t cols);
int64_t norm_grad_groups(int64_t rows, int64_t cols);

template <int DT> struct Elem;     // storage of a matrix element
template <> struct Elem<kP32> { typedef float T; };
template <> struct Elem<kPBF16> { typedef uint16_t T; };
template <> struct Elem<kPF16> { typedef uint16_t T; };

// Rows may start at any element, so wide accesses claim only the element's
// own alignment; gfx950's global memory takes them at any address.
typedef u4 u4_any __attribute__((aligned(2)));
typedef u2 u2_any __attribute__((aligned(2)));

// Eight elements as they are stored.
template <int DT> struct Raw { u4 v[DT == kP32 ? 2 : 1]; };

template <int DT>
__device__ __forceinline__ void unpack8(const uint32_t w[4], float v[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = DT == kPBF16 ? bf16_lo(w[i]) : f16_lo(w[i]);
        v[2 * i + 1] = DT == kPBF16 ? bf16_hi(w[i]) : f16_hi(w[i]);
    }
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    if (DT == kPBF16) return bf16x2_rne(a, b);
    return f16_rne(a) | (f16_rne(b) << 16);
}

// NT: the non-temporal hint, where a kernel's comment gives its measure.
template <bool NT>
__device__ __forceinline__ u4 any16(const void *p)
{
    if (NT) return sld<u4_any>(p);
    return gld<u4_any>(p);
}

template <bool NT>
__device__ __forceinline__ void put16(void *p, u4 v)
{
    if (NT) sst<u4_any>(p, v);
    else gst<u4_any>(p, v);
}

// Eight elements from p + j: `cnt` of them exist (the rest read as 0).  EIGHTS:
// cnt is 0 or 8, as where rows are a multiple of eight long; the code for
// single elements, and the registers it keeps apart, fall away.
template <int DT, bool EIGHTS = false, bool NT = false>
__device__ __forceinline__ Raw<DT> load_raw(const void *p, int64_t j, int cnt)
{
    typedef typename Elem<DT>::T T;
    const T *q = (const T *)p + j;
    Raw<DT> r;
    if (EIGHTS) {
        r.v[0] = r.v[DT == kP32] = (u4){0, 0, 0, 0};
        if (cnt > 0) {
            r.v[0] = any16<NT>(q);
            if (DT == kP32) r.v[DT == kP32] = any16<NT>(q + 4);
        }
        return r;
    }
    if (cnt >= 8) {
        r.v[0] = any16<NT>(q);
        if (DT == kP32) r.v[DT == kP32] = any16<NT>(q + 4);
        return r;
    }
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        w[i] = 0;
        if (i < cnt) w[i] = DT == kP32 ? gld<uint32_t>(q + i) : gld<uint16_t>(q + i);
    }
    if (DT == kP32) {
        r.v[0] = (u4){w[0], w[1], w[2], w[3]};
        r.v[DT == kP32] = (u4){w[4], w[5], w[6], w[7]};
    } else {
        r.v[0] = (u4){w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16};
    }
    return r;
}

template <int DT>
__device__ __forceinline__ void unpack_raw(const Raw<DT> &r, float v[8])
{
    if (DT == kP32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = bitsf(r.v[i >> 2 & (DT == kP32)][i & 3]);
    } else {
        const uint32_t w[4] = {r.v[0][0], r.v[0][1], r.v[0][2], r.v[0][3]};
        unpack8<DT>(w, v);
    }
}

// Eight values as they are stored, rounded to nearest-even.
template <int DT>
__device__ __forceinline__ Raw<DT> pack_raw(const float v[8])
{
    Raw<DT> r;
    if (DT == kP32) {
        r.v[0] = (u4){fbits(v[0]), fbits(v[1]), fbits(v[2]), fbits(v[3])};
        r.v[DT == kP32] = (u4){fbits(v[4]), fbits(v[5]), fbits(v[6]), fbits(v[7])};
    } else {
        r.v[0] = (u4){pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3]), pack2<DT>(v[4], v[5]), pack2<DT>(v[6], v[7])};
    }
    return r;
}

template <int DT, bool EIGHTS = false, bool NT = false>
__device__ __forceinline__ void load8(const void *p, int64_t j, int cnt, float v[8])
{
    unpack_raw<DT>(load_raw<DT, EIGHTS, NT>(p, j, cnt), v);
}

template <int DT, bool EIGHTS = false, bool NT = false>
__device__ __forceinline__ void store_raw(void *p, int64_t j, int cnt, const Raw<DT> &r)
{
    typedef typename Elem<DT>::T T;
    T *q = (T *)p + j;
    if (cnt >= 8) {
        put16<NT>(q, r.v[0]);
        if (DT == kP32) put16<NT>(q + 4, r.v[DT == kP32]);
        return;
    }
    if (EIGHTS) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (i < cnt) {
            if (DT == kP32) gst<uint32_t>(q + i, r.v[i >> 2 & (DT == kP32)][i & 3]);
            else gst<uint16_t>(q + i, (uint16_t)(r.v[0][i >> 1] >> (16 * (i & 1))));
        }
    }
}

template <int DT, bool EIGHTS = false, bool NT = false>
__device__ __forceinline__ void store8(void *p, int64_t j, int cnt, const float v[8])
{
    store_raw<DT, EIGHTS, NT>(p, j, cnt, pack_raw<DT>(v));
}

// The same from a matrix whose element type is known at run time (weights).
template <bool EIGHTS>
__device__ __forceinline__ void load8_any(int dt, const void *p, int64_t j, int cnt, float v[8])
{
    if (dt == kP32) load8<kP32, EIGHTS>(p, j, cnt, v);
    else if (dt == kPBF16) load8<kPBF16, EIGHTS>(p, j, cnt, v);
    else load8<kPF16, EIGHTS>(p, j, cnt, v);
}

__device__ __forceinline__ int left8(int64_t j, int64_t end) { return end - j >= 8 ? 8 : end > j ? (int)(end - j) : 0; }

__device__ __forceinline__ double two_words(uint32_t lo, uint32_t hi) { return __hiloint2double((int)hi, (int)lo); }

template <int CTRL>
__device__ __forceinline__ double dpp_add(double x)
{
    const uint32_t lo = (uint32_t)__double2loint(x), hi = (uint32_t)__double2hiint(x);
    return x + two_words((uint32_t)__builtin_amdgcn_mov_dpp((int)lo, CTRL, 0xF, 0xF, true),
                         (uint32_t)__builtin_amdgcn_mov_dpp((int)hi, CTRL, 0xF, 0xF, true));
}

// x of both lanes of a pair 16 lanes apart (within a half of the wave), 32 lanes apart.
__device__ __forceinline__ double swap16_add(double x)
{
    const uint32_t lo = (uint32_t)__double2loint(x), hi = (uint32_t)__double2hiint(x);
    const auto l = __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
    const auto h = __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
    return two_words(l[0], h[0]) + two_words(l[1], h[1]);
}

__device__ __forceinline__ double swap32_add(double x)
{
    const uint32_t lo = (uint32_t)__double2loint(x), hi = (uint32_t)__double2hiint(x);
    const auto l = __builtin_amdgcn_permlane32_swap(lo, lo, false, false);
    const auto h = __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
    return two_words(l[0], h[0]) + two_words(l[1], h[1]);
}

// Sum over 8, 16, 32 or 64 lanes, the same bits in every lane: each step adds
// two partial sums that both sides hold (lanes 1, 2, 7 - i and 15 - i away by
// DPP; then the rows and the halves of the wave by gfx950's lane swaps).
template <int LANES>
__device__ __forceinline__ double lanes_sum(double x)
{
    x = dpp_add<0xB1>(x);
    x = dpp_add<0x4E>(x);
    x = dpp_add<0x141>(x);
    if (LANES >= 16) x = dpp_add<0x140>(x);
    if (LANES >= 32) x = swap16_add(x);
    if (LANES >= 64) x = swap32_add(x);
    return x;
}

// 1/sqrt(x) to within 2^-51: the hardware's estimate and two Newton steps, a
// tenth of the instructions of a division after a square root (each of which
// every wave would run once a row: 33 -> 31 us of a pass over 8192 x 4096).
// Where a step has no value (x zero or infinite) the estimate is the result.
__device__ __forceinline__ double inverse_root(double x)
{
    const double y0 = __builtin_amdgcn_rsq(x);
    double y = y0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const double e = __builtin_fma(-x * y, y, 1.0);
        y = __builtin_fma(0.5 * y, e, y);
    }
    return y == y ? y : y0;
}

// Largest of the 16 lanes of a row (every lane ends with it): the first steps
// of wave_max_u32.
__device__ __forceinline__ uint32_t row16_max_u32(uint32_t v)
{
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x124, 0xF, 0xF, true));
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x128, 0xF, 0xF, true));
    return v;
}

__device__ __forceinline__ uint32_t abs_max8(const float v[8])
{
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, fbits(v[i]) & 0x7FFFFFFFu);
    return a;
}

// Scale byte of a block whose largest magnitude has the bits `a`: X =
// 2^(byte - 127) is the smallest power of two with A <= 448 X (448 = 1.75 *
// 2^8: the exponent of A less 8, one more if its significand passes 1.75), at
// least 2^-127; 0 for a block of zeros, 255 (NaN) if A is NaN or infinite.
__host__ __device__ inline uint32_t block_scale(uint32_t a)
{
    const int e = (int)(a >> 23) + ((a & 0x7FFFFFu) > 0x600000u ? 1 : 0) - 8;
    if (a >= 0x7F800000u) return 255u;
    return e > 0 ? (uint32_t)e : 0u;
}

// 1/X, exact: the exponent field 254 - byte is at least 6 for a finite block.
__host__ __device__ inline float block_inverse(uint32_t byte) { return bitsf((254u - byte) << 23); }

// E4M3 codes of four values times inv, nearest-even.  Every |v * inv| is at
// most 448, so the conversion never leaves the grid; the product is exact
// unless it falls below the binary32 normal range, where it codes as 0.
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inv)
{
    int w = 0;
    w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
    return (uint32_t)w;
}

__device__ __forceinline__ u2 encode8(const float v[8], uint32_t byte)
{
    if (byte == 255u) return (u2){0u, 0u};    // a NaN block's codes are zeros: its scale says NaN
    const float inv = block_inverse(byte);
    return (u2){encode4(v[0], v[1], v[2], v[3], inv), encode4(v[4], v[5], v[6], v[7], inv)};
}

// The same codes by gfx950's scaled conversions, which divide by the power of
// two X (given as a binary32 word, the scale's byte in its exponent) on the way:
// equal to encode4's on every block that is not NaN, at half its instructions.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, uint32_t x)
{
    typedef short pair __attribute__((ext_vector_type(2)));
    pair w;
    w = __builtin_nondeterministic_value(w);    // each half is written: no register is cleared first
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, a, b, bitsf(x), false);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, c, d, bitsf(x), true);
    return __builtin_bit_cast(uint32_t, w);
}

// The scale of a block whose largest magnitude has the bits `a`, as that word:
// block_scale(a) << 23 in three instructions, for a finite block (adding
// 0x1FFFFF carries into the exponent where the significand passes 1.75).
__device__ __forceinline__ uint32_t scale_word(uint32_t a)
{
    return __builtin_elementwise_sub_sat((a + 0x1FFFFFu) & 0x7F800000u, 8u << 23);
}

constexpr uint32_t kLostWord = 255u << 23;     // of a block that holds a NaN or an infinity

__device__ __forceinline__ u2 codes8(const float v[8], uint32_t word)
{
    return (u2){codes4(v[0], v[1], v[2], v[3], word), codes4(v[4], v[5], v[6], v[7], word)};
}

// Codes of eight values of a block whose largest magnitude has the bits `a`;
// word becomes its scale's.  Every lane of the wave calls it: lost blocks, whose
// codes are zeros, are looked at only where the wave has one.
__device__ __forceinline__ u2 code_block(const float v[8], uint32_t a, uint32_t &word)
{
    word = scale_word(a);
    u2 code = codes8(v, word);
    if (__any(a >= 0x7F800000u) && a >= 0x7F800000u) {
        word = kLostWord;
        code = (u2){0u, 0u};
    }
    return code;
}

// Eight values of a block-coded row, from its codes and their scale's byte:
// code times 2^(byte - 127), exact where that is a binary32 number; NaN for 255.
__device__ __forceinline__ void decode8(u2 code, uint32_t byte, float v[8])
{
    const float x = bitsf(byte << 23);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const f2_t lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(code[i], x, false);
        const f2_t hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(code[i], x, true);
        v[4 * i] = lo[0];
        v[4 * i + 1] = lo[1];
        v[4 * i + 2] = hi[0];
        v[4 * i + 3] = hi[1];
    }
}

// Bits of the largest magnitude of eight values; 0x7F800000 or more if one is
// infinite or NaN (of either sign): the maximum that propagates NaNs takes three
// operands and their magnitudes at once.
__device__ __forceinline__ float max_abs(float a, float b)
{
    return __builtin_elementwise_maximum(__builtin_fabsf(a), __builtin_fabsf(b));
}

__device__ __forceinline__ uint32_t top8(const float v[8])
{
    float m = max_abs(v[0], v[1]);
#pragma unroll
    for (int i = 2; i < 8; i += 2) m = __builtin_elementwise_maximum(m, max_abs(v[i], v[i + 1]));
    return fbits(m);
}

// A kernel's argument record where the launch left it.  A record of many
// matrices held in scalar registers spills them; read again where it is used
// (again() forgets what was read) it costs a scalar load.
#if defined(__HIP_DEVICE_COMPILE__)
#define OPT_CONST __attribute__((address_space(4)))
#else
#define OPT_CONST
#endif

template <class A>
__device__ __forceinline__ const OPT_CONST A *kernargs() { return (const OPT_CONST A *)__builtin_amdgcn_kernarg_segment_ptr(); }

template <class A>
__device__ __forceinline__ const OPT_CONST A *again(const OPT_CONST A *a)
{
#if defined(__HIP_DEVICE_COMPILE__)
    asm volatile("" : "+s"(a));
#endif
    return a;
}

__device__ __forceinline__ Codes copy(const OPT_CONST Codes &q) { return Codes{q.codes, q.ld, q.scales, q.lds}; }

// The wave's number, in a scalar register.
__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6); }

}  // namespace optstep
