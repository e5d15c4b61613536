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
// roundings: k goes through norm and rotation in fp64 (as many lanes a cycle as
// fp32 on this chip), v is taken as it is, and a quotient is looked at again
// where it is a tie.
#include <math.h>

#include "elem.hpp"
#include "launch.hpp"
#include "qmm_device.hpp"

namespace qmm {

constexpr float KV4_TOP = 57344.f;

template <typename S, bool VEC>
__device__ __forceinline__ void load8(const S *p, S (&e)[8])
{
    if constexpr (VEC) {
        const int4_t r = *reinterpret_cast<const int4_t *>(p);
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
        *reinterpret_cast<int4_t *>(p) = r;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = e[i];
    }
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

__device__ __forceinline__ float rint_(float x) { return __builtin_rintf(x); }
__device__ __forceinline__ double rint_(double x) { return __builtin_rint(x); }
__device__ __forceinline__ float fma_(float x, float y, float z) { return __builtin_fmaf(x, y, z); }
__device__ __forceinline__ double fma_(double x, double y, double z) { return __builtin_fma(x, y, z); }

// rint(x / s) for |x / s| <= 16, ties to even (inv: 1 / s, rounded).  Off a tie rint(x inv)
// is it; at one the rest x - t s is exactly s / 2 either way.
template <typename T>
__device__ __forceinline__ T quotient(T x, T s, T inv)
{
    const T t = rint_(x * inv), r = fma_(-t, s, x);
    const T even = T(2) * rint_(fma_(t, T(0.5), r > T(0) ? T(0.25) : T(-0.25)));
    return (r < T(0) ? -r : r) == T(0.5) * s ? even : t;
}

// ---------------------------------------------------------------------------
// q (and, where they go to tensors, k): bound by memory, read once and written
// once.  As in append.hip a lane owns two vectors of 8 elements that turn
// together (past rot two that stay), of HP heads of one token, so that cos and
// sin are read once for them; U lanes own a row, and the sum of its squares goes
// round them.
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
            const float r = 1.f / sqrtf(sum / (float)a.D + a.eps);
            if (live) {
                S wa[8], wb[8];
                load8<S, true>(w + first, wa);
                load8<S, true>(w + second, wb);
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
// k and v into the cache: a lane owns 8 elements in a row (a dword of codes),
// LN lanes a token's row; range and zero-point go round the G / 8 lanes of a group.  A
// workgroup takes one head of 256 / LN tokens, whose rows stand side by side in a
// page.
// ---------------------------------------------------------------------------
template <typename S, bool VEC, int LN, typename T>
__device__ __forceinline__ void put_rows(const HeadsArgs &a, int block, const S *src, int64_t ts, const S *weight, bool turn, bool pairs, uint8_t *codes,
                                         int64_t c_ps, int64_t c_ts, uint16_t *scales, int64_t s_ps)
{
    const int lane = threadIdx.x & 63, u = threadIdx.x % LN, d = 8 * u;
    const int64_t tt = (int64_t)block * (256 / LN) + threadIdx.x / LN;
    const bool in_row = d < a.D;
    const int t = (int)(tt < a.T ? tt : 0);
    const S *row = src + (int64_t)t * ts;

    T x[8];
    {
        S e[8];
        load8<S, VEC>(row + (in_row ? d : 0), e);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = in_row ? (T)to_f32(e[i]) : T(0);
    }
    if constexpr (sizeof(T) == 8) {
        T r = T(1);
        if (weight) {
            T sum = T(0);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fma_(x[i], x[i], sum);
#pragma unroll
            for (int m = 1; m < LN; m <<= 1) sum += __shfl_xor(sum, m);
            r = T(1) / sqrt(sum / (T)a.D + (T)a.eps);
        }
        auto scaled = [&](int at, T (&y)[8]) {        // y: elements of the row from `at` on
            if (!weight) return;
            S w[8];
            load8<S, true>(weight + at, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = y[i] * r * (T)to_f32(w[i]);
        };
        if (in_row) scaled(d, x);
        if (turn && d < a.rot) {
            const int pos = min(max(a.positions[t], 0), a.table_rows - 1);
            const float *line = a.rope + (size_t)pos * a.rot;
            if (pairs) {
                float cs[4], sn[4];
                load_line<4>(line + d / 2, cs);
                load_line<4>(line + a.rot / 2 + d / 2, sn);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const T p = x[2 * i], q = x[2 * i + 1];
                    x[2 * i] = p * (T)cs[i] - q * (T)sn[i];
                    x[2 * i + 1] = q * (T)cs[i] + p * (T)sn[i];
                }
            } else {
                const bool low = d < a.rot / 2;
                const int other = low ? d + a.rot / 2 : d - a.rot / 2, at = low ? d : other;
                float cs[8], sn[8];
                load_line<8>(line + at, cs);
                load_line<8>(line + a.rot / 2 + at, sn);
                S e[8];
                T y[8];
                load8<S, VEC>(row + other, e);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = (T)to_f32(e[i]);
                scaled(other, y);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = x[i] * (T)cs[i] + (low ? -y[i] : y[i]) * (T)sn[i];
            }
        }
    }

    T lo = T(0), hi = T(0);
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        nan = nan || x[i] != x[i];
        x[i] = x[i] > T(KV4_TOP) ? T(KV4_TOP) : x[i] < T(-KV4_TOP) ? T(-KV4_TOP) : x[i];
        lo = x[i] < lo ? x[i] : lo;
        hi = x[i] > hi ? x[i] : hi;
    }
    const int span = a.G / 8;
    for (int m = 1; m < span; m <<= 1) {
        const T l2 = __shfl_xor(lo, m), h2 = __shfl_xor(hi, m);
        lo = l2 < lo ? l2 : lo;
        hi = h2 > hi ? h2 : hi;
    }
    const uint64_t of_group = ((uint64_t(1) << span) - 1) << (lane & ~(span - 1));
    nan = (__ballot(nan) & of_group) != 0;

    const float s = scale_of((double)hi - (double)lo);
    const T st = (T)s, inv = T(1) / st;
    const T zq = quotient(T(0) - lo, st, inv), z = zq > T(15) ? T(15) : zq;
    uint32_t word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        T c = quotient(x[i], st, inv) + z;
        c = c < T(0) ? T(0) : c > T(15) ? T(15) : c;
        word |= (uint32_t)(int)(nan ? T(0) : c) << (4 * i);
    }
    const int64_t slot = tt < a.T ? a.slots[t] : -1;
    if (!in_row || slot < 0 || slot >= (int64_t)a.pages * a.page) return;
    const int pg = (int)slot / a.page, at = (int)slot - pg * a.page;
    *reinterpret_cast<uint32_t *>(codes + (int64_t)pg * c_ps + (int64_t)at * c_ts + d / 2) = word;
    if (u % span == 0) {
        const uint32_t sz = nan ? 0x7e00u : as_u16((_Float16)s) | (uint32_t)as_u16((_Float16)(float)z) << 16;
        *reinterpret_cast<uint32_t *>(scales + (int64_t)pg * s_ps + 2 * ((int64_t)at * (a.D / a.G) + d / a.G)) = sz;
    }
}

template <typename S, bool PAIRS, bool VEC, int U, int HP, bool STORE>
__global__ __launch_bounds__(256) void heads_kernel(const HeadsArgs a)
{
    const int groups = (a.Hq + a.Hk + HP - 1) / HP, turned = a.turn_blocks;
    if ((int)blockIdx.x < turned) {
        turn_rows<S, PAIRS, VEC, U, HP>(a, (int)blockIdx.x, groups);
        return;
    }
    if constexpr (STORE) {
        const int id = (int)blockIdx.x - turned, block = id / (2 * a.Hkv), h2 = id - block * 2 * a.Hkv;
        if (h2 < a.Hkv)
            put_rows<S, VEC, 2 * U, double>(a, block, (const S *)a.k + (int64_t)h2 * a.k_hs, a.k_ts, (const S *)a.k_weight, a.rot > 0, PAIRS,
                                            a.k_codes + (int64_t)h2 * a.kc_hs, a.kc_ps, a.kc_ts, a.k_scale + (int64_t)h2 * a.ks_hs, a.ks_ps);
        else
            put_rows<S, VEC, 2 * U, float>(a, block, (const S *)a.v + (int64_t)(h2 - a.Hkv) * a.v_hs, a.v_ts, (const S *)nullptr, false, false,
                                           a.v_codes + (int64_t)(h2 - a.Hkv) * a.vc_hs, a.vc_ps, a.vc_ts, a.v_scale + (int64_t)(h2 - a.Hkv) * a.vs_hs, a.vs_ps);
    }
}

template <typename S, bool PAIRS, bool VEC, int U, bool STORE>
static hipError_t heads_go(HeadsArgs a, hipStream_t st)
{
    constexpr int HP = 2;
    const int64_t turned = ((int64_t)a.T + 256 / U - 1) / (256 / U) * ((a.Hq + a.Hk + HP - 1) / HP);
    const int64_t put = STORE ? ((int64_t)a.T + 128 / U - 1) / (128 / U) * 2 * a.Hkv : 0;
    if ((turned + put) * 256 >= (int64_t(1) << 32)) return hipErrorNotSupported;   // threads of a launch
    if (turned + put == 0) return hipSuccess;
    a.turn_blocks = (int)turned;
    hipLaunchKernelGGL((heads_kernel<S, PAIRS, VEC, U, HP, STORE>), dim3((unsigned)(turned + put)), dim3(256), 0, st, a);
    return hipGetLastError();
}
template <typename S, bool PAIRS, bool VEC, bool STORE>
static hipError_t heads_width(const HeadsArgs &a, hipStream_t st)
{
    return a.D <= 64 ? heads_go<S, PAIRS, VEC, 4, STORE>(a, st) : a.D <= 128 ? heads_go<S, PAIRS, VEC, 8, STORE>(a, st) : heads_go<S, PAIRS, VEC, 16, STORE>(a, st);
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
// elements of a token and head.
// ---------------------------------------------------------------------------
template <typename S, bool VEC>
__global__ __launch_bounds__(256) void read4_kernel(const Read4Args a)
{
    const int per = a.D / 8;
    const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, rows = (int64_t)a.T * a.Hkv;
    const int64_t r2 = id / per;
    const int u = (int)(id - r2 * per), d = 8 * u;
    if (r2 >= 2 * rows) return;
    const bool is_k = r2 < rows;
    const int64_t r = is_k ? r2 : r2 - rows;
    const int t = (int)(r / a.Hkv), h = (int)(r - (int64_t)t * a.Hkv);
    const int64_t slot = a.slots[t];
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (slot >= 0 && slot < (int64_t)a.pages * a.page) {
        const int pg = (int)slot / a.page, at = (int)slot - pg * a.page;
        const uint8_t *codes = is_k ? a.k_codes + (int64_t)pg * a.kc_ps + (int64_t)h * a.kc_hs + (int64_t)at * a.kc_ts
                                    : a.v_codes + (int64_t)pg * a.vc_ps + (int64_t)h * a.vc_hs + (int64_t)at * a.vc_ts;
        const uint16_t *scales = (is_k ? a.k_scale + (int64_t)pg * a.ks_ps + (int64_t)h * a.ks_hs : a.v_scale + (int64_t)pg * a.vs_ps + (int64_t)h * a.vs_hs) +
                                 2 * ((int64_t)at * (a.D / a.G) + d / a.G);
        const uint32_t word = *reinterpret_cast<const uint32_t *>(codes + d / 2), sz = *reinterpret_cast<const uint32_t *>(scales);
        const float s = (float)as_half((uint16_t)sz), z = (float)as_half((uint16_t)(sz >> 16));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = ((float)((word >> (4 * i)) & 15u) - z) * s;
    }
    S *dst = is_k ? (S *)a.k_out + (int64_t)t * a.ko_ts + (int64_t)h * a.ko_hs : (S *)a.v_out + (int64_t)t * a.vo_ts + (int64_t)h * a.vo_hs;
    store8<S, VEC>(dst + d, x);
}

hipError_t launch_read4(const Read4Args &a, bool bf16, bool vec, hipStream_t st)
{
    const int64_t blocks = (2 * (int64_t)a.T * a.Hkv * (a.D / 8) + 255) / 256;
    if (blocks * 256 >= (int64_t(1) << 32)) return hipErrorNotSupported;   // threads of a launch
    const dim3 grid((unsigned)blocks);
    if (bf16) {
        if (vec) hipLaunchKernelGGL((read4_kernel<bf16_t, true>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((read4_kernel<bf16_t, false>), grid, dim3(256), 0, st, a);
    } else {
        if (vec) hipLaunchKernelGGL((read4_kernel<_Float16, true>), grid, dim3(256), 0, st, a);
        else hipLaunchKernelGGL((read4_kernel<_Float16, false>), grid, dim3(256), 0, st, a);
    }
    return hipGetLastError();
}

}  // namespace qmm
