// heads.hip -- norms of q and k for each head with their rotary positions, and a
// paged cache whose keys and values are held in 4 bits: written and read back.
//
// Norm and rotation, for every token and head of D elements:
//     y = x / sqrt(mean(x^2) + eps) * w,   (a, b) -> (a cos - b sin, b cos + a sin)
// for the pairs (i, i + rot/2), or (2i, 2i + 1), of the first rot elements, cos
// and sin from the fp32 table's row positions[t].
//
// The cache holds codes c in 0 .. 15 (element i of a token at bits 4i of its
// row) and for each G elements a scale s and a zero-point z, x = (c - z) s:
//     lo = min(0, min x), hi = max(0, max x)
//     s  = (hi - lo) / 15 to 7 significant bits, at least 2^-18
//     z  = clamp(rint(-lo / s), 0, 15),   c = clamp(rint(x / s) + z, 0, 15)
// rint to the even one of two.  c - z has 4 bits and s 7: every x of the cache
// is a number of fp16, and whoever multiplies by it rounds nothing.  x beyond
// +-57344 is stored as that (the largest (c - z) s is then 60928); a NaN makes
// its group's scale NaN.
//
// What decides between two codes must not depend on the order of a few fp32
// roundings: the codes are those of the formulas.  v is taken as it is, a quotient is
// looked at again where it is a tie, and k where fp32 leaves a doubt.
#include <math.h>

#include <type_traits>

#include "elem.hpp"
#include "launch.hpp"
#include "qmm_device.hpp"

namespace qmm {

constexpr float KV4_TOP = 57344.f;

// Rows are read once and written once: neither leaves a trace in the caches (8192 tokens of
// 64 heads of 128 normed and turned: 57 us with the default policy, 54 so; with k and v into the cache
// and read back from it 76 and 72).
template <typename S, bool VEC>
__device__ __forceinline__ void load8(const S *p, S (&e)[8])
{
    if constexpr (VEC) {
        const int4_t r = __builtin_nontemporal_load(reinterpret_cast<const int4_t *>(p));
        __builtin_memcpy(e, &r, sizeof r);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = p[i];
    }
}
template <typename S, bool VEC>
__device__ __forceinline__ void store8(S *p, const float (&x)[8])
{
    S e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = from_f32<S>(x[i]);
    if constexpr (VEC) {
        int4_t r;
        __builtin_memcpy(&r, e, sizeof r);
        __builtin_nontemporal_store(r, reinterpret_cast<int4_t *>(p));
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = e[i];
    }
}
template <typename S>
__device__ __forceinline__ void load_weights(const S *p, S (&e)[8])
{
    const int4_t r = *reinterpret_cast<const int4_t *>(p);
    __builtin_memcpy(e, &r, sizeof r);
}
template <int N>
__device__ __forceinline__ void load_line(const float *p, float (&x)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float4_t r = *reinterpret_cast<const float4_t *>(p + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[i + e] = r[e];
    }
}

// (hi - lo) / 15 to 7 significant bits, ties to even: the fp32 quotient says between
// which two it lies (or, one of them too low, is itself next to the upper one), their
// middle times 15 is exact.
__device__ __forceinline__ float scale_of(double range)
{
    float f = (float)(range * (1.0 / 15.0));
    f = f < 0x1p-19f ? 0x1p-19f : f;
    const uint32_t b = __builtin_bit_cast(uint32_t, f), low = b & ~0x1ffffu;
    const double half = 0x1p-7 * (double)__builtin_bit_cast(float, b & 0x7f800000u);
    const double mid = 15.0 * ((double)__builtin_bit_cast(float, low) + half);
    const bool up = range > mid || (range == mid && (low & 0x20000u));
    return fmaxf(__builtin_bit_cast(float, low + (up ? 0x20000u : 0u)), 0x1p-18f);
}

// rint(x / s) for |x / s| <= 16, ties to even (inv: 1 / s, rounded).  Off a tie rint(x inv)
// is it; at one the rest x - t s is exactly s / 2 either way.
__device__ __forceinline__ double quotient(double x, double s, double inv)
{
    const double t = __builtin_rint(x * inv), r = __builtin_fma(-t, s, x);
    const double even = 2.0 * __builtin_rint(__builtin_fma(t, 0.5, r > 0.0 ? 0.25 : -0.25));
    return __builtin_fabs(r) == 0.5 * s ? even : t;
}

// ---------------------------------------------------------------------------
// q (and, where they go to tensors, k): bound by memory, read once and written
// once.  As in append.hip a lane owns two vectors of 8 elements that turn
// together (past rot two that stay), of HP heads of one token, so that cos and
// sin are read once for them; U lanes own a row, and the sum of its squares goes
// round them (of smaller or larger numbers where it leaves fp32).  8192 tokens of 64 + 8
// heads of 128, bf16: 59 us, 5.2 TB/s (a large copy the same); 1 token 4.2, the call.
// ---------------------------------------------------------------------------
template <typename S, bool PAIRS, bool VEC, int U, int HP>
__device__ __forceinline__ void turn_rows(const HeadsArgs &a, int block, int groups)
{
    const int heads = a.Hq + a.Hk, tb = block / groups, h0 = (block - tb * groups) * HP;
    const int64_t tt = (int64_t)tb * (256 / U) + threadIdx.x / U;
    const int u = threadIdx.x % U;
    const bool live = tt < a.T && 16 * u < a.D;
    const int t = (int)(tt < a.T ? tt : 0);
    const bool turns = 16 * u < a.rot;
    const int first = PAIRS || !turns ? 16 * u : 8 * u;
    const int second = PAIRS || !turns ? first + 8 : first + a.rot / 2;

    float cs[8], sn[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        cs[i] = 1.f;
        sn[i] = 0.f;
    }
    if (turns) {
        const int pos = min(max(a.positions[t], 0), a.table_rows - 1);
        const float *line = a.rope + (size_t)pos * a.rot + 8 * u;
        load_line<8>(line, cs);
        load_line<8>(line + a.rot / 2, sn);
    }

    S raw[HP][2][8];
#pragma unroll
    for (int i = 0; i < HP; ++i) {
        const int h = h0 + i;
#pragma unroll
        for (int e = 0; e < 8; ++e) raw[i][0][e] = raw[i][1][e] = (S)0.f;
        if (h < heads && live) {
            const S *src = h < a.Hq ? (const S *)a.q + (int64_t)t * a.q_ts + (int64_t)h * a.q_hs
                                    : (const S *)a.k + (int64_t)t * a.k_ts + (int64_t)(h - a.Hq) * a.k_hs;
            load8<S, VEC>(src + first, raw[i][0]);
            load8<S, VEC>(src + second, raw[i][1]);
        }
    }
#pragma unroll
    for (int i = 0; i < HP; ++i) {
        const int h = h0 + i;
        if (h >= heads) break;
        float x[2][8];
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int e = 0; e < 8; ++e) x[p][e] = to_f32(raw[i][p][e]);
        const S *w = (const S *)(h < a.Hq ? a.q_weight : a.k_weight);
        if (w) {
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += x[0][e] * x[0][e] + x[1][e] * x[1][e];
#pragma unroll
            for (int m = 1; m < U; m <<= 1) sum += __shfl_xor(sum, m);
            float mean = sum / (float)a.D + (float)a.eps;
            if (__any(!(mean > 0x1p-100f && mean < 0x1p112f))) {
                // squares (or eps) outside fp32's range: the same of x 2^-up and eps 4^-up, the larger about 1
                float top = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, fmaxf(fabsf(x[0][e]), fabsf(x[1][e])));
#pragma unroll
                for (int m = 1; m < U; m <<= 1) top = fmaxf(top, __shfl_xor(top, m));
                const int half = a.eps > 0.0 ? (__builtin_amdgcn_frexp_exp(a.eps) + 1) >> 1 : -1000;
                const int up = top > 0.f ? max(__builtin_amdgcn_frexp_expf(top), half) : half;
                sum = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[0][e] = ldexpf(x[0][e], -up);
                    x[1][e] = ldexpf(x[1][e], -up);
                    sum += x[0][e] * x[0][e] + x[1][e] * x[1][e];
                }
#pragma unroll
                for (int m = 1; m < U; m <<= 1) sum += __shfl_xor(sum, m);
                mean = sum / (float)a.D + (float)ldexp(a.eps, -2 * up);
            }
            const float r = 1.f / sqrtf(mean);
            if (live) {
                S wa[8], wb[8];
                load_weights(w + first, wa);
                load_weights(w + second, wb);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[0][e] = x[0][e] * r * to_f32(wa[e]);
                    x[1][e] = x[1][e] * r * to_f32(wb[e]);
                }
            }
        }
        if (!live) continue;
        if (turns) {
            float y[2][8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // neighbouring form: pair e is elements 2e, 2e + 1 of the 16 in a row
                const float p = PAIRS ? x[e / 4][2 * (e % 4)] : x[0][e], q = PAIRS ? x[e / 4][2 * (e % 4) + 1] : x[1][e];
                const float yp = p * cs[e] - q * sn[e], yq = q * cs[e] + p * sn[e];
                if constexpr (PAIRS) {
                    y[e / 4][2 * (e % 4)] = yp;
                    y[e / 4][2 * (e % 4) + 1] = yq;
                } else {
                    y[0][e] = yp;
                    y[1][e] = yq;
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[0][e] = y[0][e];
                x[1][e] = y[1][e];
            }
        }
        S *dst = h < a.Hq ? (S *)a.q_out + (int64_t)t * a.qo_ts + (int64_t)h * a.qo_hs
                          : (S *)a.k_out + (int64_t)t * a.ko_ts + (int64_t)(h - a.Hq) * a.ko_hs;
        store8<S, VEC>(dst + first, x[0]);
        store8<S, VEC>(dst + second, x[1]);
    }
}

// ---------------------------------------------------------------------------
// k and v into the cache: a lane owns 8 elements in a row (a dword of codes) of KP
// heads, k and v of each, LN lanes a token's row; range and zero-point go round the G / 8
// lanes of a group.  A workgroup's 256 / LN tokens stand side by side in a page's head.  Its
// waves wait for memory (one row a wave: 31 us for 8192 tokens of 2 x 8 heads, k and v of two
// heads 26; few tokens: see heads_pick), so they run between q's, which is bound by memory: 68 us
// for both, 54 for q's 64 heads alone (4.6 TB/s; on inputs that the last-level cache holds 64).
//
// k is normed, turned and mapped in fp32 first, with a bound of what its roundings may have
// moved its elements by; where that leaves a scale, a zero-point or a code in doubt
// (a few waves in a hundred) the wave does it again in fp64.  (All of it in fp64: 41 us
// for k and v alone, row by row.)
// ---------------------------------------------------------------------------
template <typename S> struct Row4 {
    S own[8], other[8];         // this lane's elements; those that turn with them (halves)
    S w_own[8], w_other[8];
    float cs[8], sn[8];         // pairs: four of each
    float turn;                 // the largest of them, at least 1
    bool norm, turns, pairs, low;
};

// f over `span` lanes side by side (4, 8, 16 or 32; the same in all of them)
template <typename F>
__device__ __forceinline__ float round_lanes(float x, int span, F f)
{
    auto moved = [](float v, auto ctrl) { return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), decltype(ctrl)::value, 0xf, 0xf, true)); };
    x = f(x, moved(x, std::integral_constant<int, 0xb1>()));                   // lane ^ 1
    x = f(x, moved(x, std::integral_constant<int, 0x4e>()));                   // lane ^ 2
    if (span >= 8) x = f(x, moved(x, std::integral_constant<int, 0x141>()));   // 7 - lane of 8
    if (span >= 16) x = f(x, moved(x, std::integral_constant<int, 0x140>()));  // 15 - lane of 16
    if (span >= 32) x = f(x, __shfl_xor(x, 16));
    return x;
}

// The row's elements after norm and rotation in fp32.  Returns a bound of what its roundings move any of
// this lane's 8 by, 16 of 2^-24 of |x| + |y|; infinity where the sum of squares leaves fp32's range.  They are 12.75 at
// most: 8 + log2(LN) <= 13 of the sum, as the lanes add it (eight in a row, then a tree: another order needs another
// bound), a division, eps and its rounding, halved by the root; root, reciprocal; 2 of the rotation; the product.  (w x is exact.)
template <int LN, typename S>
__device__ __forceinline__ float turned8(const HeadsArgs &a, const Row4<S> &r, float (&x)[8])
{
    float root = 1.f, size = 0.f, y[8];
    bool in_range = true;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = to_f32(r.own[i]);
    if (r.norm) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
        sum = round_lanes(sum, LN, [](float p, float q) { return p + q; });
        const float mean = sum / (float)a.D + (float)a.eps;
        in_range = mean > 0x1p-100f && mean < 0x1p112f;
        root = 1.f / sqrtf(mean);
#pragma unroll
        for (int i = 0; i < 8; ++i) {        // (products of two 16-bit numbers are exact)
            x[i] *= to_f32(r.w_own[i]);
            size = fmaxf(size, fabsf(x[i]));
        }
    }
    if (r.turns && r.pairs) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float p = x[2 * i], q = x[2 * i + 1];
            x[2 * i] = p * r.cs[i] - q * r.sn[i];
            x[2 * i + 1] = q * r.cs[i] + p * r.sn[i];
            size = fmaxf(size, fabsf(p) + fabsf(q));
        }
    } else if (r.turns) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y[i] = to_f32(r.other[i]);
            if (r.norm) y[i] *= to_f32(r.w_other[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            size = fmaxf(size, fabsf(x[i]) + fabsf(y[i]));
            x[i] = x[i] * r.cs[i] + (r.low ? -y[i] : y[i]) * r.sn[i];
        }
    }
    if (r.norm) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= root;
    }
    return in_range ? 0x1p-20f * size * root * r.turn : INFINITY;
}
// The same in fp64.
template <int LN, typename S>
__device__ __forceinline__ void turned8(const HeadsArgs &a, const Row4<S> &r, double (&x)[8])
{
    double root = 1.0;
    if (r.norm) {
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += (double)to_f32(r.own[i]) * (double)to_f32(r.own[i]);
        for (int m = 1; m < LN; m <<= 1) sum += __shfl_xor(sum, m);
        root = 1.0 / sqrt(sum / (double)a.D + a.eps);
    }
    auto scaled = [&](S v, S w) { return r.norm ? (double)to_f32(v) * (double)to_f32(w) * root : (double)to_f32(v); };
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = scaled(r.own[i], r.w_own[i]);
    if (r.turns && r.pairs) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const double p = x[2 * i], q = x[2 * i + 1];
            x[2 * i] = p * (double)r.cs[i] - q * (double)r.sn[i];
            x[2 * i + 1] = q * (double)r.cs[i] + p * (double)r.sn[i];
        }
    } else if (r.turns) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const double q = scaled(r.other[i], r.w_other[i]);
            x[i] = x[i] * (double)r.cs[i] + (r.low ? -q : q) * (double)r.sn[i];
        }
    }
}

// Scale, zero-point and codes of a lane's 8 elements in their group of `span` lanes.  x is off by at
// most `err` (in some lane of the group); false: that leaves a doubt.  Exact elements (err 0) leave none:
//     y = x / s, corrected by its rest once, is the quotient where fp32 has it, so ties are ties
//     (s has 7 bits, x at most 11: off a tie the quotient is 2^-13 of it away).
__device__ __forceinline__ bool map8(float (&x)[8], float err, int span, float &s, float &z, uint32_t &word)
{
    float lo = 0.f, hi = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = __builtin_amdgcn_fmed3f(x[i], -KV4_TOP, KV4_TOP);
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
    }
    lo = round_lanes(lo, span, [](float p, float q) { return fminf(p, q); });
    hi = round_lanes(hi, span, [](float p, float q) { return fmaxf(p, q); });
    const double range = (double)hi - (double)lo;
    s = scale_of(range);
    bool sure = true;
    if (__any(err > 0.f)) {
        err = round_lanes(err, span, [](float p, float q) { return fmaxf(p, q); });
        sure = scale_of(range - 2.0 * (double)err) == scale_of(range + 2.0 * (double)err);
    }
    const float inv = __builtin_amdgcn_rcpf(s), limit = err > 0.f ? 0.5f * s - err : INFINITY;
    auto nearest = [&](float v) {
        float y = v * inv;
        y = fmaf(fmaf(-y, s, v), inv, y);
        const float t = __builtin_rintf(y);
        sure = sure && fabsf(fmaf(-t, s, v)) < limit;
        return t;
    };
    z = fminf(nearest(0.f - lo), 15.f);
    float c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = __builtin_amdgcn_fmed3f(nearest(x[i]) + z, 0.f, 15.f);
    const float low = fmaf(fmaf(fmaf(c[3], 16.f, c[2]), 16.f, c[1]), 16.f, c[0]), high = fmaf(fmaf(fmaf(c[7], 16.f, c[6]), 16.f, c[5]), 16.f, c[4]);
    word = (uint32_t)low | (uint32_t)high << 16;
    return sure;
}
__device__ __forceinline__ void map8(double (&x)[8], int span, float &s, float &z, uint32_t &word)
{
    double lo = 0.0, hi = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = x[i] > (double)KV4_TOP ? (double)KV4_TOP : x[i] < -(double)KV4_TOP ? -(double)KV4_TOP : x[i];
        lo = x[i] < lo ? x[i] : lo;
        hi = x[i] > hi ? x[i] : hi;
    }
    for (int m = 1; m < span; m <<= 1) {
        const double l2 = __shfl_xor(lo, m), h2 = __shfl_xor(hi, m);
        lo = l2 < lo ? l2 : lo;
        hi = h2 > hi ? h2 : hi;
    }
    s = scale_of(hi - lo);
    const double inv = 1.0 / (double)s, zq = quotient(0.0 - lo, (double)s, inv), zt = zq > 15.0 ? 15.0 : zq;
    z = (float)zt;
    word = 0;
    for (int i = 0; i < 8; ++i) {
        double c = quotient(x[i], (double)s, inv) + zt;
        c = c < 0.0 ? 0.0 : c > 15.0 ? 15.0 : c;
        word |= (uint32_t)(int)(c == c ? c : 0.0) << (4 * i);
    }
}

// HP heads of a token, k and v of each: all that is read is on its way before the first is mapped.
template <typename S, bool PAIRS, bool VEC, int LN, int HP>
__device__ __forceinline__ void put_rows(const HeadsArgs &a, int block, int h0)
{
    const int lane = threadIdx.x & 63, u = threadIdx.x % LN, d = 8 * u;
    const int64_t tt = (int64_t)block * (256 / LN) + threadIdx.x / LN;
    const bool in_row = d < a.D;
    const int t = (int)(tt < a.T ? tt : 0), from = in_row ? d : 0;
    const int64_t slot = tt < a.T ? a.slots[t] : -1;

    Row4<S> r;
    r.norm = a.k_weight != nullptr;
    r.turns = d < a.rot;
    r.pairs = PAIRS;
    r.low = d < a.rot / 2;
    r.turn = 1.f;
    const int other = PAIRS || !r.turns ? from : r.low ? d + a.rot / 2 : d - a.rot / 2;
    const int pos = a.rot > 0 ? min(max(a.positions[t], 0), a.table_rows - 1) : 0;
    S k[HP][8], k_other[HP][8], v[HP][8];
#pragma unroll
    for (int i = 0; i < HP; ++i) {
        const int h = min(h0 + i, a.Hkv - 1);
        const S *row = (const S *)a.k + (int64_t)t * a.k_ts + (int64_t)h * a.k_hs;
        load8<S, VEC>(row + from, k[i]);
        if (!PAIRS && r.turns) load8<S, VEC>(row + other, k_other[i]);
        load8<S, VEC>((const S *)a.v + (int64_t)t * a.v_ts + (int64_t)h * a.v_hs + from, v[i]);
    }
    if (r.norm) {
        load_weights((const S *)a.k_weight + from, r.w_own);
        if (!PAIRS && r.turns) load_weights((const S *)a.k_weight + other, r.w_other);
    }
    if (r.turns) {
        const float *line = a.rope + (size_t)pos * a.rot + (PAIRS ? d / 2 : r.low ? d : other);
        load_line<4>(line, reinterpret_cast<float(&)[4]>(r.cs[0]));
        load_line<4>(line + a.rot / 2, reinterpret_cast<float(&)[4]>(r.sn[0]));
        if constexpr (!PAIRS) {
            load_line<4>(line + 4, reinterpret_cast<float(&)[4]>(r.cs[4]));
            load_line<4>(line + a.rot / 2 + 4, reinterpret_cast<float(&)[4]>(r.sn[4]));
        }
#pragma unroll
        for (int i = 0; i < (PAIRS ? 4 : 8); ++i) r.turn = fmaxf(r.turn, fmaxf(fabsf(r.cs[i]), fabsf(r.sn[i])));
    }

    const int span = a.G / 8;
    const uint64_t of_group = ((uint64_t(1) << span) - 1) << (lane & ~(span - 1));
    const bool live = in_row && slot >= 0 && slot < (int64_t)a.pages * a.page;
    const int pg = live ? a.by_page((int)slot) : 0, at = live ? (int)slot - pg * a.page : 0;
#pragma unroll
    for (int i = 0; i < HP; ++i) {
        const int h = h0 + i;
        if (h >= a.Hkv) break;
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            float x[8], s, z, err = 0.f;
            uint32_t word;
            bool nan = false;
            if (side == 0) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    r.own[e] = in_row ? k[i][e] : (S)0.f;
                    r.other[e] = k_other[i][e];
                }
                err = turned8<LN>(a, r, x);
                if (!r.norm && a.rot == 0) err = 0.f;
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = in_row ? to_f32(v[i][e]) : 0.f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) nan = nan || x[e] != x[e];
            const bool sure = map8(x, err, span, s, z, word);
            if (side == 0 && __any(!sure)) {
                double y[8];
                turned8<LN>(a, r, y);
                nan = false;
#pragma unroll
                for (int e = 0; e < 8; ++e) nan = nan || y[e] != y[e];
                map8(y, span, s, z, word);
            }
            nan = (__ballot(nan) & of_group) != 0;
            if (!live) continue;
            uint8_t *codes = side == 0 ? a.k_codes + (int64_t)pg * a.kc_ps + (int64_t)h * a.kc_hs + (int64_t)at * a.kc_ts
                                       : a.v_codes + (int64_t)pg * a.vc_ps + (int64_t)h * a.vc_hs + (int64_t)at * a.vc_ts;
            *reinterpret_cast<uint32_t *>(codes + d / 2) = nan ? 0u : word;
            if (u % span == 0) {
                uint16_t *scales = (side == 0 ? a.k_scale + (int64_t)pg * a.ks_ps + (int64_t)h * a.ks_hs : a.v_scale + (int64_t)pg * a.vs_ps + (int64_t)h * a.vs_hs) +
                                   2 * ((int64_t)at * a.by_G(a.D) + a.by_G(d));
                *reinterpret_cast<uint32_t *>(scales) = nan ? 0x7e00u : as_u16((_Float16)s) | (uint32_t)as_u16((_Float16)z) << 16;
            }
        }
    }
}

// KP: heads of k and v that a lane takes (0: no cache)
template <typename S, bool PAIRS, bool VEC, int U, int HP, int KP>
__global__ __launch_bounds__(256) void heads_kernel(const HeadsArgs a)
{
    const int groups = (a.Hq + a.Hk + HP - 1) / HP, id = (int)blockIdx.x;
    if constexpr (KP == 0) {
        turn_rows<S, PAIRS, VEC, U, HP>(a, id, groups);
    } else {
        // every by_period.d-th workgroup takes k or v: computing and moving run side by side
        const int nth = a.by_period(id);
        if (nth >= a.put_blocks || nth * a.by_period.d != id) {
            turn_rows<S, PAIRS, VEC, U, HP>(a, id - min(nth + 1, a.put_blocks), groups);
            return;
        }
        const int kv_groups = (a.Hkv + KP - 1) / KP, block = nth / kv_groups;
        put_rows<S, PAIRS, VEC, 2 * U, KP>(a, block, (nth - block * kv_groups) * KP);
    }
}

template <typename S, bool PAIRS, bool VEC, int U, int KP>
static hipError_t heads_go(HeadsArgs a, hipStream_t st)
{
    constexpr int HP = 2;
    const int64_t turned = ((int64_t)a.T + 256 / U - 1) / (256 / U) * ((a.Hq + a.Hk + HP - 1) / HP);
    int64_t put = 0;
    if constexpr (KP > 0) put = ((int64_t)a.T + 128 / U - 1) / (128 / U) * ((a.Hkv + KP - 1) / KP);
    if ((turned + put) * 256 >= (int64_t(1) << 32)) return hipErrorNotSupported;   // threads of a launch
    if (turned + put == 0) return hipSuccess;
    if (KP > 0) {
        a.put_blocks = (int)put;
        a.by_period.set((turned + put) / put);
        a.by_page.set(a.page);
        a.by_G.set(a.G);
    }
    hipLaunchKernelGGL((heads_kernel<S, PAIRS, VEC, U, HP, KP>), dim3((unsigned)(turned + put)), dim3(256), 0, st, a);
    return hipGetLastError();
}
template <typename S, bool PAIRS, bool VEC, int U, bool STORE>
static hipError_t heads_pick(const HeadsArgs &a, hipStream_t st)
{
    if constexpr (!STORE) {
        return heads_go<S, PAIRS, VEC, U, 0>(a, st);
    } else {
        // One head a lane is soonest done where all workgroups run at once, two move more where they go in rounds
        // (32 + 2 x 8 heads of 128, us, one and two: 1 token 4.3 and 6.1, 256: 6.1 and 8.0, 2048: 16.2 and 17.0,
        // 4096 with 64 heads of q: 37.1 and 36.6, 8192: 67 and 64).
        return (int64_t)a.T * a.Hkv * 2 * U <= 1024 * 256 ? heads_go<S, PAIRS, VEC, U, 1>(a, st) : heads_go<S, PAIRS, VEC, U, 2>(a, st);
    }
}
template <typename S, bool PAIRS, bool VEC, bool STORE>
static hipError_t heads_width(const HeadsArgs &a, hipStream_t st)
{
    return a.D <= 64 ? heads_pick<S, PAIRS, VEC, 4, STORE>(a, st) : a.D <= 128 ? heads_pick<S, PAIRS, VEC, 8, STORE>(a, st) : heads_pick<S, PAIRS, VEC, 16, STORE>(a, st);
}
template <typename S, bool STORE>
static hipError_t heads_type(const HeadsArgs &a, bool vec, hipStream_t st)
{
    if (a.pairs) return vec ? heads_width<S, true, true, STORE>(a, st) : heads_width<S, true, false, STORE>(a, st);
    return vec ? heads_width<S, false, true, STORE>(a, st) : heads_width<S, false, false, STORE>(a, st);
}

// vec: every row stands at a multiple of 16 bytes.  store: k and v go to the cache (a.Hk is 0).
hipError_t launch_heads(const HeadsArgs &a, bool bf16, bool vec, bool store, hipStream_t st)
{
    if (bf16) return store ? heads_type<bf16_t, true>(a, vec, st) : heads_type<bf16_t, false>(a, vec, st);
    return store ? heads_type<_Float16, true>(a, vec, st) : heads_type<_Float16, false>(a, vec, st);
}

// ---------------------------------------------------------------------------
// Tokens of the cache as 16-bit rows: bound by what it writes.  A lane takes 8
// elements of a token, of HP heads and both sides; U lanes a row.  A workgroup's
// tokens stand side by side in a page's head, its heads side by side in a
// token's output.  131072 tokens of 2 x 8 heads of 128, G 64: 128 to 136 us, 5.1 to 5.4 TB/s, four fifths of it written;
// 1001 of 2 x 4 heads of 96: 5.6, the call.
// ---------------------------------------------------------------------------
template <typename S, bool VEC, int U, int HP>
__global__ __launch_bounds__(256) void read4_kernel(const Read4Args a)
{
    const int hg = (a.Hkv + HP - 1) / HP, tb = (int)blockIdx.x / hg, h0 = ((int)blockIdx.x - tb * hg) * HP;
    const int64_t tt = (int64_t)tb * (256 / U) + threadIdx.x / U;
    const int u = threadIdx.x % U, d = 8 * u;
    if (tt >= a.T || d >= a.D) return;
    const int t = (int)tt;
    const int64_t slot = a.slots[t];
    const bool live = slot >= 0 && slot < (int64_t)a.pages * a.page;
    const int pg = live ? a.by_page((int)slot) : 0, at = live ? (int)slot - pg * a.page : 0;
    const uint8_t *codes[2] = {a.k_codes + (int64_t)pg * a.kc_ps + (int64_t)at * a.kc_ts + d / 2, a.v_codes + (int64_t)pg * a.vc_ps + (int64_t)at * a.vc_ts + d / 2};
    const int s_at = 2 * (at * (a.D >> a.lg_G) + (d >> a.lg_G));
    const uint16_t *scales[2] = {a.k_scale + (int64_t)pg * a.ks_ps + s_at, a.v_scale + (int64_t)pg * a.vs_ps + s_at};
    S *out[2] = {(S *)a.k_out + (int64_t)t * a.ko_ts + d, (S *)a.v_out + (int64_t)t * a.vo_ts + d};
    const int64_t c_hs[2] = {a.kc_hs, a.vc_hs}, s_hs[2] = {a.ks_hs, a.vs_hs}, o_hs[2] = {a.ko_hs, a.vo_hs};

    uint32_t word[HP][2], sz[HP][2];
#pragma unroll
    for (int i = 0; i < HP; ++i)
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const int h = min(h0 + i, a.Hkv - 1);
            word[i][p] = *reinterpret_cast<const uint32_t *>(codes[p] + h * c_hs[p]);
            sz[i][p] = *reinterpret_cast<const uint32_t *>(scales[p] + h * s_hs[p]);
        }
#pragma unroll
    for (int i = 0; i < HP; ++i) {
        const int h = h0 + i;
        if (h >= a.Hkv) break;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const float s = (float)as_half((uint16_t)sz[i][p]), z = (float)as_half((uint16_t)(sz[i][p] >> 16));
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = live ? ((float)((word[i][p] >> (4 * e)) & 15u) - z) * s : 0.f;
            store8<S, VEC>(out[p] + h * o_hs[p], x);
        }
    }
}

template <typename S, bool VEC, int U>
static hipError_t read4_go(const Read4Args &a, hipStream_t st)
{
    constexpr int HP = 4;
    const int64_t blocks = ((int64_t)a.T + 256 / U - 1) / (256 / U) * ((a.Hkv + HP - 1) / HP);
    if (blocks * 256 >= (int64_t(1) << 32)) return hipErrorNotSupported;   // threads of a launch
    hipLaunchKernelGGL((read4_kernel<S, VEC, U, HP>), dim3((unsigned)blocks), dim3(256), 0, st, a);
    return hipGetLastError();
}
template <typename S, bool VEC>
static hipError_t read4_width(const Read4Args &a, hipStream_t st)
{
    return a.D <= 64 ? read4_go<S, VEC, 8>(a, st) : a.D <= 128 ? read4_go<S, VEC, 16>(a, st) : read4_go<S, VEC, 32>(a, st);
}
hipError_t launch_read4(const Read4Args &a, bool bf16, bool vec, hipStream_t st)
{
    if (bf16) return vec ? read4_width<bf16_t, true>(a, st) : read4_width<bf16_t, false>(a, st);
    return vec ? read4_width<_Float16, true>(a, st) : read4_width<_Float16, false>(a, st);
}

}  // namespace qmm
