// opt_kernels_heads.hip -- the norm of queries and keys for each head with the
// rotation by position in the same pass, and its backward pass.
//
// Forward, for each head x of dim elements:  r = fl(1/sqrt(mean(x^2) + eps)),
// n = x r w, and the first rot elements turn in pairs (a, b) by the angle whose
// cosine c and sine s the position's row of the table holds: (a c - b s,
// b c + a s).  Backward: dn is dy turned the other way, g = dn w, k = r^2
// mean(g x), dx = r (g - x k), dw = sum over tokens and heads of dn (x r).
//
// A head stays in the registers of L lanes, eight consecutive elements each; a
// wave holds 64/L heads (a unit) of one token.  What an element takes of itself
// and of its pair's other half, A = w c and B = w' (+-)s with the partner's
// weight w', is the same for all of a token's heads and formed once for them:
// y = (x r) A + (x' r) B.
//
// Bound by HBM and by the latency of a wave's chain (position, table's row and
// elements, sums, root).  A pass among others over 8192 tokens of 32 + 8 heads of
// 128, bf16: forward with codes 41 us (215 MB, 5.3 TB/s; the vector units are busy
// 55 % of the time), without 35; backward from codes 49 us (214 MB, 4.4 TB/s; 66 %),
// of which the sums of both weights' gradients are 4.  Stores carry the
// non-temporal hint (51.7 us forward without); so do the loads where no codes are
// written (43.8 -> 37.9 us; with codes 43.9 -> 45.7) and the backward pass's (53.1
// -> 51.1).
#include "opt_pass.h"

namespace optstep {

// How a pair's other element is found.  kHalves: pairs (i, i + rot/2) with
// rot/2 and dim multiples of eight (or no pairs): a lane's partners are another
// lane's eight.  kWhole: the same where the head fills its lanes (dim = 8 L), so
// that no lane's loads are masked.  kNear: pairs (2 i, 2 i + 1), dim a multiple
// of eight: a lane's own.  kAny: what is left, element by element.
enum { kWhole = 0, kHalves = 1, kNear = 2, kAny = 3 };
constexpr bool by_halves(int mode) { return mode <= kHalves; }

// A token's row of the table; null if its position has none.
__device__ __forceinline__ const float *table_row(const HeadTurn &t, int64_t token)
{
    int64_t p = token;
    if (t.positions)       // the token is the wave's: a scalar load
        p = t.wide_positions ? ((const OPT_CONST int64_t *)t.positions)[token] : (int64_t)((const OPT_CONST int32_t *)t.positions)[token];
    if (p < 0 || p >= t.table_rows) return nullptr;
    return t.table + p * t.ldt;
}

// Where an element of the first rot has its partner, whether it is a pair's
// first, and which pair that is.
struct Pair { int partner, index; bool first; };

template <int MODE>
__device__ __forceinline__ Pair pair_of(const HeadTurn &t, int e)
{
    const int h = t.rot / 2;
    if (MODE == kNear || (MODE == kAny && t.neighbours)) return Pair{e ^ 1, e >> 1, !(e & 1)};
    return Pair{e < h ? e + h : e - h, e < h ? e : e - h, e < h};
}

// Whether element c + i turns (rot and c are even: the two of a pair of
// neighbours alike, so that half as many masks are kept).
__device__ __forceinline__ bool turns(const HeadTurn &t, int c, int i) { return c + (i & ~1) < t.rot; }

// cos and sin of the eight elements from c on, the sine with the sign of what
// the partner adds (BACK: turned the other way); 1 and 0 where nothing turns.
template <int MODE, bool BACK>
__device__ __forceinline__ void angles(const HeadTurn &t, const float *row, int c, float cs[8], float sn[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        cs[i] = 1.0f;
        sn[i] = 0.0f;
    }
    if (!row || c >= t.rot) return;
    if (by_halves(MODE)) {
        const Pair p = pair_of<MODE>(t, c);
        load8<kP32, true>(row + p.index, 0, 8, cs);
        load8<kP32, true>(row + t.rot / 2 + p.index, 0, 8, sn);
#pragma unroll
        for (int i = 0; i < 8; ++i) sn[i] = p.first != BACK ? -sn[i] : sn[i];
        return;
    }
    // all loads at once: elements that do not turn read the row's first
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool on = turns(t, c, i);
        const Pair p = pair_of<MODE>(t, on ? c + i : 0);
        const float x = gld<float>(row + p.index), y = gld<float>(row + t.rot / 2 + p.index);
        cs[i] = on ? x : 1.0f;
        sn[i] = on ? (p.first != BACK ? -y : y) : 0.0f;
    }
}

__device__ __forceinline__ float load_any(int dt, const void *p, int64_t j)
{
    if (dt == kP32) return gld<float>((const float *)p + j);
    const uint32_t b = gld<uint16_t>((const uint16_t *)p + j);
    return dt == kPBF16 ? bf16_lo(b) : f16_lo(b);
}

// The weights of the eight elements from c on, and (PARTNERS) of their partners
// (1 where nothing turns: an infinite weight keeps to its own element).
template <int MODE, bool PARTNERS>
__device__ __forceinline__ void weights(const HeadTurn &t, const void *w, int c, int cnt, float v[8], float vp[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = vp[i] = 1.0f;
    if (!w) return;
    load8_any<MODE != kAny>(t.w_dtype, w, c, cnt, v);
    if (!PARTNERS || c >= t.rot) return;
    if (by_halves(MODE)) {
        load8_any<true>(t.w_dtype, w, pair_of<MODE>(t, c).partner, cnt, vp);
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool on = turns(t, c, i);
        const float x = MODE == kNear ? v[i ^ 1] : load_any(t.w_dtype, w, on ? pair_of<MODE>(t, c + i).partner : 0);
        vp[i] = on ? x : 1.0f;
    }
}

// Where element `at` of a wave's 512 lies in the LDS: eight apart in every lane,
// no two lanes share a bank.
__device__ __forceinline__ int wave_at(int at) { return at + (at >> 6); }
constexpr int kWaveFloats = 512 + 8;

// The partners of a lane's eight elements of a head; zeros where nothing turns,
// so that an infinity or a NaN there keeps to its own element (its partner's
// angle is 0, but infinity times 0 is NaN).  Every lane of the wave calls it;
// `lds` is the wave's own (kAny).
template <int DT, int MODE>
__device__ __forceinline__ void partners(const HeadTurn &t, const Raw<DT> &raw, int c, float v[8], float *lds)
{
    const int lane = threadIdx.x & 63, h = t.rot / 2;
    if (by_halves(MODE)) {
        // the lane h/8 up or down the head; what it holds, as stored
        const int from = 4 * (c >= t.rot ? lane : c < h ? lane + h / 8 : lane - h / 8);
        Raw<DT> o;
#pragma unroll
        for (int j = 0; j < (DT == kP32 ? 2 : 1); ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o.v[j][i] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)raw.v[j][i]);
        if (t.rot < t.dim && c >= t.rot) {         // (whole rotations skip it)
#pragma unroll
            for (int j = 0; j < (DT == kP32 ? 2 : 1); ++j) o.v[j] = (u4){0u, 0u, 0u, 0u};
        }
        unpack_raw<DT>(o, v);
        return;
    }
    unpack_raw<DT>(raw, v);
    if (MODE == kNear || t.neighbours) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float x = v[i];
            v[i] = turns(t, c, i) ? v[i + 1] : 0.0f;
            v[i + 1] = turns(t, c, i) ? x : 0.0f;
        }
        return;
    }
    // by element through the LDS, whose accesses of one wave keep their order
#pragma unroll
    for (int i = 0; i < 8; ++i) lds[wave_at(8 * lane + i)] = v[i];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int e = c + i, d = e >= t.rot ? 0 : e < h ? h : -h;
        const float x = lds[wave_at(8 * lane + i + d)];
        v[i] = turns(t, c, i) ? x : 0.0f;
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ HeadTurn turn_of(const OPT_CONST HeadTurn &t)
{
    return HeadTurn{t.tokens, t.table_rows, t.ldt, t.table, t.positions, t.dim, t.rot, t.wide_positions, t.neighbours, t.w_dtype, t.eps, t.inv_dim};
}

// A forward launch's arguments.
struct HeadLaunch { HeadArgs a; int per; };

// Largest over the lanes that share one 128-element block.
template <int L>
__device__ __forceinline__ uint32_t block_max_u32(uint32_t v)
{
    if (L >= 16) return row16_max_u32(v);
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));
    return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));
}

__device__ __forceinline__ float root_of(double ss, const HeadTurn &t) { return (float)inverse_root(__builtin_fma(ss, t.inv_dim, t.eps)); }

// Loads of a unit's lanes: a head past the last reads the last one's elements
// (kWhole) or none.
template <int DT, int MODE, bool NT>
__device__ __forceinline__ Raw<DT> load_head(const char *p, int c, int cnt)
{
    if (MODE == kWhole) return load_raw<DT, true, NT>(p, c, 8);
    return load_raw<DT, MODE != kAny, NT>(p, c, cnt);
}

// Ends when the loads of x have arrived.  A wave asks for all its heads at once
// and waits here once: the hardware counts loads and stores together, so that a
// load waited for after a store waits for the store too.
template <int DT, int N>
__device__ __forceinline__ void arrived(Raw<DT> (&x)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        asm volatile("" : "+v"(x[i].v[0]));
        if (DT == kP32) asm volatile("" : "+v"(x[i].v[DT == kP32]));
    }
}

constexpr int kHeadThreads = 256;

// Units a wave takes at most: their elements are in its registers at once (at
// 8192 tokens of 32 + 8 heads of 128, ten units a token: 3 measured 48.8 us, 4
// 43.1, 5 42.1, 6 43.1).
template <int DT> constexpr int head_most() { return DT == kP32 ? 3 : 5; }

// A wave takes `per` units of a token, of the queries and then of the keys, all
// of whose elements it asks for first.
template <int DT, int L, int MODE, bool CODES>
__global__ __launch_bounds__(kHeadThreads) void head_norm_kernel(HeadArgs, int)
{
    constexpr int S = 64 / L, kSize = sizeof(typename Elem<DT>::T), kMost = head_most<DT>();
    __shared__ float lds[MODE == kAny ? kHeadThreads / 64 * kWaveFloats : 1];
    const OPT_CONST HeadLaunch *k = kernargs<HeadLaunch>();
    const HeadTurn t = turn_of(k->a.t);
    const int per = k->per, lane = threadIdx.x % L, c = 8 * lane, slot = (threadIdx.x & 63) / L;
    const int cnt = left8(c, t.dim);
    const int headsq = (int)k->a.s[0].heads, headsk = (int)k->a.s[1].heads;
    const int unitsq = (headsq + S - 1) / S, units = unitsq + (headsk + S - 1) / S, parts = (units + per - 1) / per;
    const int64_t waves = t.tokens * parts, step = (int64_t)gridDim.x * (kHeadThreads / 64);
    for (int64_t w = (int64_t)blockIdx.x * (kHeadThreads / 64) + wave_id(); w < waves; w += step) {
        const int64_t token = parts == 1 ? w : w < (int64_t)1 << 31 ? (uint32_t)w / (uint32_t)parts : w / parts;
        const int first = (int)(w - token * parts) * per, n = units - first < per ? units - first : per;
        // past the last head of a set: kWhole does that head's work again, to the same places
        auto head_of = [&](int u, bool keys) {
            const int head = (u - (keys ? unitsq : 0)) * S + slot, heads = keys ? headsk : headsq;
            return MODE == kWhole && head >= heads ? heads - 1 : head;
        };
        Raw<DT> raw[kMost];
#pragma unroll
        for (int j = 0; j < kMost; ++j)
            if (j < n) {
                const bool keys = first + j >= unitsq;
                const OPT_CONST HeadSet *h = k->a.s + keys;
                const int head = head_of(first + j, keys);
                const char *x = (const char *)h->x + token * h->xt * kSize + head * (h->xh * kSize);
                raw[j] = load_head<DT, MODE, !CODES>(x, c, head < (keys ? headsk : headsq) ? cnt : 0);
            }
        const float *row = t.rot ? table_row(t, token) : nullptr;
        const bool lost = t.rot && !row;            // a position the table does not hold: NaN
        float A[2][8], B[2][8], cs[8], sn[8];
        angles<MODE, false>(t, row, c, cs, sn);
#pragma unroll
        for (int set = 0; set < 2; ++set) {
            if (set ? first + n <= unitsq : first >= unitsq) continue;
            weights<MODE, true>(t, k->a.s[set].w, c, cnt, A[set], B[set]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                A[set][i] *= cs[i];
                B[set][i] *= sn[i];
            }
        }
        arrived(raw);
        const OPT_CONST HeadSet *h = k->a.s;
#pragma unroll
        for (int j = 0; j < kMost; ++j) {
            if (j >= n) break;
            const bool keys = first + j >= unitsq;
            h = again(k)->a.s + keys;
            if (first + j == unitsq || (j == 0 && keys))
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    A[0][i] = A[1][i];
                    B[0][i] = B[1][i];
                }
            const int head = head_of(first + j, keys), heads = keys ? headsk : headsq;
            const bool live = head < heads;
            const int have = MODE == kWhole ? 8 : live ? cnt : 0;
            float v[8], vp[8], o[8];
            unpack_raw<DT>(raw[j], v);
            partners<DT, MODE>(t, raw[j], c, vp, lds + wave_id() * kWaveFloats);
            double ss = 0.0;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = __builtin_fma((double)v[i], (double)v[i], ss);
            float r = root_of(lanes_sum<L>(ss), t);
            if (lost) r = bitsf(0x7FC00000u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // an infinite r (a head of tiny elements) times the zero of an element that does not turn: NaN
                const float rp = turns(t, c, by_halves(MODE) ? 0 : i) ? r : 0.0f;
                o[i] = __builtin_fmaf(vp[i] * rp, B[0][i], (v[i] * r) * A[0][i]);
            }
            store8<DT, MODE != kAny, true>((char *)h->y + token * h->yt * kSize + head * (h->yh * kSize), c, have, o);
            if (CODES && h->q.codes) {
                const Codes q = copy(h->q);
                uint32_t word;
                const u2 code = code_block(v, block_max_u32<L>(top8(v)), word);
                const int64_t line = token * heads + head;
                if (MODE == kWhole || (live && c < ((t.dim + 15) & ~15))) sst<u2>(q.codes + line * q.ld + c, code);
                if (MODE == kWhole || (have > 0 && (lane & 15) == 0)) gst<uint8_t>(q.scales + (c / kCodeBlock) * q.lds + line, (uint8_t)(word >> 23));
            }
        }
    }
}

// The backward pass: a wave takes tokens in turn.  A lane's sums of both weights'
// gradients run in binary32 over the units it has in registers at once, four at
// most, and join binary64 sums of its own in the LDS there (in registers they
// would cost a wave a SIMD).
constexpr int kHeadGradThreads = 256;
// Four waves a SIMD, which kWhole's registers allow (512 measured 72 us against 55
// at the sizes above); the other forms hold three at once.
constexpr int64_t kHeadGradGroups = 1024;

// A lane's inputs of one head, as they are stored.
template <int DT, bool CODED> struct HeadIn { Raw<DT> dy, x; };
template <int DT> struct HeadIn<DT, true> { Raw<DT> dy; u2 x; uint32_t byte; };

template <int DT, int N>
__device__ __forceinline__ void arrived(HeadIn<DT, false> (&x)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        asm volatile("" : "+v"(x[i].dy.v[0]), "+v"(x[i].x.v[0]));
        if (DT == kP32) asm volatile("" : "+v"(x[i].dy.v[DT == kP32]), "+v"(x[i].x.v[DT == kP32]));
    }
}

template <int DT, int N>
__device__ __forceinline__ void arrived(HeadIn<DT, true> (&x)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) {
        asm volatile("" : "+v"(x[i].dy.v[0]), "+v"(x[i].x), "+v"(x[i].byte));
        if (DT == kP32) asm volatile("" : "+v"(x[i].dy.v[DT == kP32]));
    }
}

constexpr int kSumRow = 72;        // 64 lanes' sums and a gap: eight rows fall into different banks by pairs

template <int DT> constexpr int head_grad_most() { return DT == kP32 ? 2 : 4; }

template <int DT, int L, int MODE, bool CODED>
__global__ __launch_bounds__(kHeadGradThreads) void head_norm_grad_kernel(HeadGradArgs)
{
    constexpr int kWaves = kHeadGradThreads / 64, S = 64 / L, kSize = sizeof(typename Elem<DT>::T), kMost = head_grad_most<DT>();
    __shared__ double comb[kWaves][2][8][kSumRow];     // a lane's sums of its columns 8 (l % L) + i
    __shared__ float lds[MODE == kAny ? kWaves * kWaveFloats : 1];
    const OPT_CONST HeadGradArgs *k = kernargs<HeadGradArgs>();
    const HeadTurn t = turn_of(k->t);
    const int lane = threadIdx.x % L, c = 8 * lane, slot = (threadIdx.x & 63) / L;
    const int cnt = left8(c, t.dim);
    const int wave = wave_id();
    const bool sums = k->part != nullptr;
    double *const mine = &comb[wave][0][0][threadIdx.x & 63];
    if (sums)
#pragma unroll
        for (int i = 0; i < 16; ++i) mine[kSumRow * i] = 0.0;
    const int64_t step = (int64_t)gridDim.x * kWaves;
    const int headsq = (int)k->s[0].heads, headsk = (int)k->s[1].heads;
    const int unitsq = (headsq + S - 1) / S, units = unitsq + (headsk + S - 1) / S;
    const int parts = (units + kMost - 1) / kMost, per = (units + parts - 1) / parts;
    float wq[8], wk[8], none[8];
    weights<MODE, false>(t, k->s[0].w, c, cnt, wq, none);
    weights<MODE, false>(t, k->s[1].w, c, cnt, wk, none);
    for (int64_t token = (int64_t)blockIdx.x * kWaves + wave_id(); token < t.tokens; token += step) {
        float cs[8], sn[8];
        bool lost = false;
#pragma unroll 1
        for (int first = 0; first < units; first += per) {
            const int n = units - first < per ? units - first : per;
            // past the last head of a set: kWhole does that head's work again, to the same places
            auto head_of = [&](int u, bool keys) {
                const int head = (u - (keys ? unitsq : 0)) * S + slot, heads = keys ? headsk : headsq;
                return MODE == kWhole && head >= heads ? heads - 1 : head;
            };
            HeadIn<DT, CODED> in[kMost];
#pragma unroll
            for (int j = 0; j < kMost; ++j)
                if (j < n) {
                    const bool keys = first + j >= unitsq;
                    const OPT_CONST HeadGradSet *h = k->s + keys;
                    const int head = head_of(first + j, keys), heads = keys ? headsk : headsq, have = head < heads ? cnt : 0;
                    in[j].dy = load_head<DT, MODE, true>((const char *)h->dy + token * h->dyt * kSize + head * (h->dyh * kSize), c, have);
                    if constexpr (CODED) {
                        const Codes q = copy(h->q);
                        const int64_t line = token * heads + head;
                        in[j].x = (u2){0u, 0u};
                        in[j].byte = 0;
                        if (MODE == kWhole || have > 0) {
                            in[j].x = gld<u2>(q.codes + line * q.ld + c);
                            in[j].byte = gld<uint8_t>(q.scales + (c / kCodeBlock) * q.lds + line);
                        }
                    } else {
                        in[j].x = load_head<DT, MODE, true>((const char *)h->x + token * h->xt * kSize + head * (h->xh * kSize), c, have);
                    }
                }
            if (first == 0) {
                const float *row = t.rot ? table_row(t, token) : nullptr;
                lost = t.rot && !row;
                angles<MODE, true>(t, row, c, cs, sn);
            }
            arrived(in);
            float dw[2][8] = {};
            const OPT_CONST HeadGradSet *h = k->s;
#pragma unroll
            for (int j = 0; j < kMost; ++j) {
                if (j >= n) break;
                const bool keys = first + j >= unitsq;
                h = again(k)->s + keys;
                const int head = head_of(first + j, keys);
                const bool live = (first + j - (keys ? unitsq : 0)) * S + slot < (keys ? headsk : headsq);
                const int have = MODE == kWhole ? 8 : live ? cnt : 0;
                float v[8], d[8], dp[8], g[8], o[8];
                unpack_raw<DT>(in[j].dy, d);
                partners<DT, MODE>(t, in[j].dy, c, dp, lds + wave_id() * kWaveFloats);
                if constexpr (CODED) {
                    decode8(in[j].x, in[j].byte, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (MODE == kAny && i >= have) v[i] = 0.0f;     // a scale that says NaN makes NaNs of the padding
                } else {
                    unpack_raw<DT>(in[j].x, v);
                }
                double ss[2] = {0.0, 0.0};
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    d[i] = __builtin_fmaf(dp[i], sn[i], d[i] * cs[i]);
                    g[i] = d[i] * (keys ? wk[i] : wq[i]);
                    const double xd = (double)v[i];
                    ss[0] = __builtin_fma(xd, xd, ss[0]);
                    ss[1] = __builtin_fma((double)g[i], xd, ss[1]);
                }
                float r = root_of(lanes_sum<L>(ss[0]), t);
                if (lost) r = bitsf(0x7FC00000u);
                const float m = (float)((double)r * (double)r * (lanes_sum<L>(ss[1]) * t.inv_dim));
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[i] *= r;
                    o[i] = __builtin_fmaf(-v[i], m, r * g[i]);
                }
                store8<DT, MODE != kAny, true>((char *)h->dx + token * h->dxt * kSize + head * (h->dxh * kSize), c, have, o);
                if (live) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (keys) dw[1][i] = __builtin_fmaf(d[i], v[i], dw[1][i]);
                        else dw[0][i] = __builtin_fmaf(d[i], v[i], dw[0][i]);
                    }
                }
            }
            // the lane's own sums: an addition in the LDS, of which nothing is waited for
#pragma unroll
            for (int q = 0; q < 2; ++q)
                if (sums && (q ? first + n > unitsq : first < unitsq))
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        __hip_atomic_fetch_add(mine + kSumRow * (8 * q + i), (double)dw[q][i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        }
    }
    if (!sums) return;
    // the workgroup's sums, over the lanes that hold the same columns, in a fixed order
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * t.dim; e += kHeadGradThreads) {
        const int q = e >= t.dim, j = e - q * t.dim;
        double v = 0.0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
#pragma unroll
            for (int l = 0; l < 64; l += L) v += comb[w][q][j & 7][(j >> 3) + l];
        gst<double>(k->part + ((int64_t)blockIdx.x * 2 + q) * t.dim + j, v);
    }
}

// dw[c] (+)= sum over the groups' partials, in binary64 and a fixed order: 16
// columns a workgroup, 64 quarter-waves every 64th group each (2 x 128 columns of
// 1024 groups: 4.9 us; 32 columns 5.6).
__global__ __launch_bounds__(1024) void head_dw_kernel(const double *part, int64_t groups, int dim, float *dwq, float *dwk, int accumulate)
{
    __shared__ double s[64][16];
    const int lane = threadIdx.x % 16, rank = threadIdx.x / 16;
    const int e = (int)blockIdx.x * 16 + lane;
    double v = 0.0;
    if (e < 2 * dim) {
#pragma unroll 16
        for (int64_t g = rank; g < groups; g += 64) v += gld<double>(part + g * 2 * dim + e);
    }
    s[rank][lane] = v;
    __syncthreads();
    if (rank == 0 && e < 2 * dim) {
        float *dw = e < dim ? dwq : dwk;
        if (!dw) return;
        const int j = e < dim ? e : e - dim;
        for (int i = 1; i < 64; ++i) v += s[i][lane];
        if (accumulate) v += (double)gld<float>(dw + j);
        gst<float>(dw + j, (float)v);
    }
}

// ---- launches --------------------------------------------------------------

static int head_lanes(int dim) { return dim <= 64 ? 8 : dim <= 128 ? 16 : dim <= 256 ? 32 : 64; }

static int mode_of(const HeadTurn &t)
{
    if (t.dim % 8 != 0) return kAny;
    if (t.rot > 0 && t.neighbours) return kNear;
    return t.rot % 16 != 0 ? kAny : t.dim == 8 * head_lanes(t.dim) ? kWhole : kHalves;
}

int64_t head_grad_groups(int64_t tokens)
{
    constexpr int kWaves = kHeadGradThreads / 64;
    const int64_t n = (tokens + kWaves - 1) / kWaves;
    return n < kHeadGradGroups ? n : kHeadGradGroups;
}

template <int DT, int L>
static hipError_t launch_head_t(const HeadArgs &a, hipStream_t st)
{
    constexpr int64_t kUnit = 64 / L, kMost = head_most<DT>();
    const int64_t units = (a.s[0].heads + kUnit - 1) / kUnit + (a.s[1].heads + kUnit - 1) / kUnit;
    int64_t per = (units + (units + kMost - 1) / kMost - 1) / ((units + kMost - 1) / kMost);     // as few parts as can be, alike
    if (per > a.t.tokens * units / 8192) per = a.t.tokens * units / 8192;                          // but waves that fill the chip
    per = per < 1 ? 1 : per;
    const int64_t waves = a.t.tokens * ((units + per - 1) / per), want = (waves + kHeadThreads / 64 - 1) / (kHeadThreads / 64);
    const unsigned grid = (unsigned)(want < (1 << 20) ? want : 1 << 20);
    const bool codes = a.s[0].q.codes || a.s[1].q.codes;
#define X(M) \
    case M: \
        if (codes) hipLaunchKernelGGL((head_norm_kernel<DT, L, M, true>), dim3(grid), dim3(kHeadThreads), 0, st, a, (int)per); \
        else hipLaunchKernelGGL((head_norm_kernel<DT, L, M, false>), dim3(grid), dim3(kHeadThreads), 0, st, a, (int)per); \
        break;
    switch (mode_of(a.t)) { X(kWhole) X(kHalves) X(kNear) X(kAny) }
#undef X
    return hipGetLastError();
}

template <int DT, int L, bool CODED>
static hipError_t launch_head_grad_t(const HeadGradArgs &a, hipStream_t st)
{
    const unsigned grid = (unsigned)head_grad_groups(a.t.tokens);
    switch (mode_of(a.t)) {
    case kWhole: hipLaunchKernelGGL((head_norm_grad_kernel<DT, L, kWhole, CODED>), dim3(grid), dim3(kHeadGradThreads), 0, st, a); break;
    case kHalves: hipLaunchKernelGGL((head_norm_grad_kernel<DT, L, kHalves, CODED>), dim3(grid), dim3(kHeadGradThreads), 0, st, a); break;
    case kNear: hipLaunchKernelGGL((head_norm_grad_kernel<DT, L, kNear, CODED>), dim3(grid), dim3(kHeadGradThreads), 0, st, a); break;
    default: hipLaunchKernelGGL((head_norm_grad_kernel<DT, L, kAny, CODED>), dim3(grid), dim3(kHeadGradThreads), 0, st, a);
    }
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
    const int64_t groups = any ? head_grad_groups(a.t.tokens) : 0;
    hipLaunchKernelGGL(head_dw_kernel, dim3((unsigned)((2 * a.t.dim + 15) / 16)), dim3(1024), 0, st, (const double *)a.part, groups, a.t.dim, dwq, dwk,
                       accumulate);
    return hipGetLastError();
}

}  // namespace optstep
