// attend4.hip -- attention of new tokens over a paged cache of 4-bit codes.
//
//     o_i = sum_j p_ij v_j,   p_ij = exp(x_ij - max_j x_ij) / sum_j exp(..),   x_ij = scale q_i . k_j
//
// over the keys j that row i sees: j <= L - n + i (L keys in the sequence, n of
// them new), and with a window j > L - n + i - window or j < sinks.  Keys and
// values are (c - z) s, c a code of 4 bits, s and z of its group of G elements.
// A row that sees no key gives zeros and a log sum of -inf.
//
// The products run on f16 matrix instructions whatever q's type.  A code becomes
// an f16 by its place in 0x6400 | c, the number 1024 + c (or 1024 + 16 c, one place
// further up): with z and 1024 taken off and times s, a scale of 7 significant bits
// gives an f16 without a rounding (one of more bits rounds once).  bf16 rows
// of q are brought to f16's range by a power of two for each row: nothing of their 8
// bits is lost down to 2^-28 of the row's largest, beyond that 2^-39 of it.
//
// The places that a block of rows looks at are numbered through: first the sinks
// (up to a multiple of `unit`), then the keys from the block's first window on.
#include <algorithm>
#include <math.h>

#include "attend.hpp"

namespace qmm {

typedef _Float16 f16_t;

// fp16 probabilities are scaled by 2^15: in full down to 2^-29 of a row's largest.
constexpr float A4_TOP = 15.f;

struct Range4 {
    int t0, n, L;
    int lo, hi;        // keys that some row sees: [lo, hi), and those below sk
    int sk;
    int start;         // lo brought down to a multiple of 16
    int S;             // places of the sinks: place v < S is key v, others key v - S + start
    int len;           // places
};
__device__ __forceinline__ Range4 range4(const Attend4Args &a, int b, int rb)
{
    Range4 r;
    int t0 = a.cu_q[b], n = a.cu_q[b + 1] - t0;
    if (t0 < 0 || n < 0 || t0 + (int64_t)n > a.T) n = 0;
    n = min(n, a.max_q);
    r.t0 = t0;
    r.n = n;
    r.L = (int)min((int64_t)max(a.kv_lens[b], 0), min((int64_t)a.width * a.page, (int64_t)a.max_kv));
    const int first = rb * a.rows / a.g, last = (min((rb + 1) * a.rows, n * a.g) - 1) / a.g;
    r.hi = max(0, min(r.L, r.L - n + last + 1));
    r.lo = a.window > 0 ? max(0, r.L - n + first - a.window + 1) : 0;
    r.sk = min(a.sinks, r.hi);
    r.start = r.lo & ~15;
    r.S = (r.sk + a.unit - 1) / a.unit * a.unit;
    if (r.S >= r.start) {              // they meet: one stretch
        r.S = 0;
        if (r.sk > 0) r.start = 0;
    }
    r.len = r.S + max(0, r.hi - r.start);
    return r;
}
__device__ __forceinline__ int key_at(const Range4 &r, int v) { return v < r.S ? v : v - r.S + r.start; }

// Whether row `i` of sequence b sees a key that stands on a page.
__device__ __forceinline__ bool row_sees(const Attend4Args &a, int b, const Range4 &kr, int i)
{
    const int hi = min(kr.L, kr.L - kr.n + i + 1), lo = a.window > 0 ? hi - a.window : 0;
    return sees_key(a, b, lo, hi) || sees_key(a, b, 0, min(min(a.sinks, lo), hi));
}

// What turns a product into a base-2 exponent: positive, or NaN as it is given.
__device__ __forceinline__ float above_zero(float x) { return x < 1e-37f ? 1e-37f : x; }

// Four dwords of q's 8 elements: f16 in codes' order (elements 0 4, 1 5, 2 6, 3 7).
__device__ __forceinline__ int4_t code_order(int4_t q)
{
    int4_t r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        r[2 * i] = (int)__builtin_amdgcn_perm((uint32_t)q[2 + i], (uint32_t)q[i], 0x05040100u);
        r[2 * i + 1] = (int)__builtin_amdgcn_perm((uint32_t)q[2 + i], (uint32_t)q[i], 0x07060302u);
    }
    return r;
}
__device__ __forceinline__ float largest(int4_t q, bf16_t)
{
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max((uint32_t)q[i] << 16 & 0x7fffffffu, (uint32_t)q[i] & 0x7fff0000u));
    return __builtin_bit_cast(float, m);
}
__device__ __forceinline__ int4_t to_f16(int4_t q, int up)     // bf16 -> f16 times 2^up
{
    int4_t r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float x = __builtin_bit_cast(float, (uint32_t)q[i] << 16), y = __builtin_bit_cast(float, (uint32_t)q[i] & 0xffff0000u);
        r[i] = pack2(ldexpf(x, up), ldexpf(y, up), f16_t());
    }
    return r;
}
// the power that brings a row whose largest is m below 2^15
__device__ __forceinline__ int rise_of(float m)
{
    return m > 0.f && m < INFINITY ? 15 - __builtin_amdgcn_frexp_expf(m) : 0;
}

// what is taken off 1024 + c and off 64 + c, and the scale, of two halves
struct Zero {
    half2_t low, high, s;
};
__device__ __forceinline__ Zero zero_of(uint32_t sc0, uint32_t sc1)
{
    Zero r;
    const half2_t z = as_half2(__builtin_amdgcn_perm(sc1, sc0, 0x07060302u));
    r.s = as_half2(__builtin_amdgcn_perm(sc1, sc0, 0x05040100u));
    r.low = half2_t{(f16_t)-1024.f, (f16_t)-1024.f} - z;
    r.high = half2_t{(f16_t)-64.f, (f16_t)-64.f} - z;
    return r;
}
// codes at bits 0 .. 3 and 16 .. 19 of w (HIGH: 4 .. 7 and 20 .. 23) as f16
template <bool HIGH>
__device__ __forceinline__ int value2(uint32_t w, const Zero &z)
{
    half2_t x = as_half2(qmm_and_or(w, HIGH ? 0x00f000f0u : 0x000f000fu, 0x64006400u));
    if constexpr (HIGH)
        x = __builtin_elementwise_fma(x, half2_t{(f16_t)0.0625f, (f16_t)0.0625f}, z.high);
    else
        x = x + z.low;
    return (int)as_u32(x * z.s);
}
// 8 codes of a dword, in codes' order
__device__ __forceinline__ int4_t values8(uint32_t w, const Zero &z)
{
    return int4_t{value2<false>(w, z), value2<true>(w, z), value2<false>(w >> 8, z), value2<true>(w >> 8, z)};
}

// ---------------------------------------------------------------------------
// Few query rows for each key head (decode, short chunks): as attend_rows_kernel, a
// workgroup takes one (sequence, key head, block of 16 QT rows, split of the
// places), its waves take blocks of 32 places in turn, each with its own running
// softmax, and are joined in LDS.
//   S^T = K Q^T   lane (g, c) holds a slice of key c's codes: with DP = 128, 32 elements from 32 g
//                 on, 16 bytes, one group's scale; q stands in the same order.
//   O^T = V^T P^T lane (g, c) holds 8 elements of 8 keys (4g .. 4g + 3 of either half), a dword
//                 each; two keys' dwords are put together before the codes are taken out, so that a
//                 pair of f16 is one element of two keys.
// ---------------------------------------------------------------------------
__host__ __device__ constexpr int rows4_occupancy(int DP, int QT) { return DP <= 128 && QT == 1 ? 3 : 2; }

template <typename S, int DP, bool P16, int QT, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(rows4_occupancy(DP, QT), rows4_occupancy(DP, QT)))) void attend4_rows_kernel(const Attend4Args a)
{
    constexpr int KJ = DP / 32;                          // steps of Q K^T
    constexpr int KW = DP == 64 ? 2 : 4;                 // dwords of a slice
    constexpr int KL = DP / (32 * KW);                   // slices of a lane
    constexpr int VW = DP >= 128 ? 8 : 4;                // codes of a V row in one load
    constexpr int VC = DP / (16 * VW);                   // loads of a V row
    constexpr int XT = DP / 16;                          // O^T tiles
    constexpr int LD = DP + 4;                           // row pitch of the join in LDS
    extern __shared__ __attribute__((aligned(16))) float att_lds[];

    int id = blockIdx.x;
    const int groups = a.B * a.Hkv, bh = id % groups;
    id /= groups;
    const int rb = id % a.rblocks, split = id / a.rblocks, b = bh / a.Hkv, hk = bh - b * a.Hkv;

    const Range4 kr = range4(a, b, rb);
    const int nrow = min(16 * QT, kr.n * a.g - rb * a.rows);     // live rows
    if (nrow <= 0) return;
    const int begin = split * a.chunk, end = min(kr.len, begin + a.chunk);
    if (begin >= end && split > 0) return;

    const int lane = threadIdx.x & 63, wave = wave_id(), g = lane >> 4, c = lane & 15;
    const S tag = (S)0.f;

    int4_t q[QT][KJ];
    int vhi[QT], vlo[QT];      // the row's keys: [vlo, vhi), and those below the sinks
    float sl[QT];
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        const int r = rb * a.rows + 16 * qt + c;
        const int i = r / a.g, hq = hk * a.g + (r - i * a.g);
        const bool live = 16 * qt + c < nrow;
        vhi[qt] = live ? kr.L - kr.n + i + 1 : 0;
        vlo[qt] = a.window > 0 ? vhi[qt] - a.window : 0;
        const char *row = (const char *)a.q + (int64_t)(kr.t0 + (live ? i : 0)) * a.q_ts + (int64_t)(live ? hq : 0) * a.q_hs;
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
            const int d = 32 * KW * (j / KW) + 8 * KW * g + 8 * (j % KW);
            q[qt][j] = *reinterpret_cast<const int4_t *>(row + (d < a.D ? 2 * d : 0));
            if (!live || d >= a.D) q[qt][j] = int4_t{0, 0, 0, 0};
            if constexpr (!__is_same(S, f16_t)) top = fmaxf(top, largest(q[qt][j], tag));
        }
        sl[qt] = a.scale * ATT_LOG2E;
        if constexpr (!__is_same(S, f16_t)) {
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const int up = rise_of(top);
#pragma unroll
            for (int j = 0; j < KJ; ++j) q[qt][j] = to_f16(q[qt][j], up);
            sl[qt] = ldexpf(sl[qt], -up);
        }
        sl[qt] = above_zero(sl[qt]);
#pragma unroll
        for (int j = 0; j < KJ; ++j) q[qt][j] = code_order(q[qt][j]);
    }
    // keys that every row of the block sees: [all_lo, all_hi) (and those below the sinks)
    const int all_hi = min(kr.hi, kr.L - kr.n + rb * a.rows / a.g + 1);
    const int all_lo = a.window > 0 ? kr.hi - a.window : 0;

    uint32_t koff[KL], ksoff[KL], voff[VC], vsoff[VC];
    bool kin[KL], vin[VC];
#pragma unroll
    for (int j = 0; j < KL; ++j) {
        const int d = 32 * KW * j + 8 * KW * g;
        kin[j] = d < a.D;
        koff[j] = P16 ? (kin[j] ? (uint32_t)c * a.k_ts + d / 2 : ATT_OOB) : (kin[j] ? d / 2 : 0);
        ksoff[j] = P16 ? (kin[j] ? (uint32_t)c * a.s_ts + 4 * (d >> a.lg_G) : ATT_OOB) : (kin[j] ? 4 * (d >> a.lg_G) : 0);
    }
#pragma unroll
    for (int x = 0; x < VC; ++x) {
        const int d = 16 * VW * x + VW * c;
        vin[x] = d < a.D;
        voff[x] = P16 ? (vin[x] ? 4u * g * a.v_ts + d / 2 : ATT_OOB) : (vin[x] ? d / 2 : 0);
        vsoff[x] = P16 ? (vin[x] ? 4u * g * a.s_ts + 4 * (d >> a.lg_G) : ATT_OOB) : (vin[x] ? 4 * (d >> a.lg_G) : 0);
    }

    const uint8_t *kbase = a.k + (int64_t)hk * a.k_hs, *vbase = a.v + (int64_t)hk * a.v_hs;
    const uint8_t *ksbase = (const uint8_t *)a.ks + (int64_t)hk * a.ks_hs, *vsbase = (const uint8_t *)a.vs + (int64_t)hk * a.vs_hs;
    const int32_t *table = a.table + (int64_t)b * a.table_s;

    // page of (each half of) block blk: P16 two uniform ids, else the id of place lane % 32
    struct Ids {
        int p[2];
    };
    auto ids_of = [&](int blk) {
        Ids r;
        const int v = begin + 32 * blk;
        if constexpr (P16) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int kk = __builtin_amdgcn_readfirstlane(key_at(kr, max(0, min(v + 16 * h, end - 1))));
                r.p[h] = table[key_page(a, kk)];
            }
        } else {
            r.p[0] = table[key_page(a, key_at(kr, max(0, min(v + (lane & 31), end - 1))))];
            r.p[1] = 0;
        }
        return r;
    };
    auto is_page = [&](int pid) { return (uint32_t)pid < (uint32_t)a.pages; };

    uint32_t kd[2][KL][KW], ksd[2][KL], vd[8][VC], vsd[8][VC];
    auto load_k = [&](int blk, const Ids &ids) {
        const int v = begin + 32 * blk;
        if constexpr (P16) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int vv = __builtin_amdgcn_readfirstlane(v + 16 * t), pid = __builtin_amdgcn_readfirstlane(ids.p[t]);
                const bool ok = vv < end && is_page(pid);
                const int kk = key_at(kr, vv), at = ok ? kk - key_page(a, kk) * a.page : 0, live = min(16, end - vv);
                const int64_t pg = ok ? pid : 0;
                const __amdgpu_buffer_rsrc_t r = make_rsrc(kbase + pg * a.k_ps + (int64_t)at * a.k_ts, ok ? (uint32_t)(live - 1) * a.k_ts + (uint32_t)a.D / 2 : 0u);
                const __amdgpu_buffer_rsrc_t rs = make_rsrc(ksbase + pg * a.ks_ps + (int64_t)at * a.s_ts, ok ? (uint32_t)live * a.s_ts : 0u);
#pragma unroll
                for (int j = 0; j < KL; ++j) {
                    ksd[t][j] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rs, ksoff[j], 0, 0);
                    load_dwords<LOAD_DEFAULT>(r, koff[j], kd[t][j], KW);
                }
            }
        } else {
            const bool there = v + (lane & 31) < end && is_page(ids.p[0]);
            const int kk = key_at(kr, max(0, min(v + (lane & 31), end - 1))), at = kk - key_page(a, kk) * a.page, pg = there ? ids.p[0] : 0;
            const int64_t off = (int64_t)pg * a.k_ps + (int64_t)at * a.k_ts, soff = (int64_t)pg * a.ks_ps + (int64_t)at * a.s_ts;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                auto from = [&](int64_t x) {
                    const uint32_t lo = (uint32_t)__shfl((int)(uint32_t)x, 16 * t + c), hi = (uint32_t)__shfl((int)(x >> 32), 16 * t + c);
                    return (int64_t)(((uint64_t)hi << 32) | lo);
                };
                const uint8_t *row = kbase + from(off), *srow = ksbase + from(soff);
#pragma unroll
                for (int j = 0; j < KL; ++j) {
                    ksd[t][j] = *reinterpret_cast<const uint32_t *>(srow + ksoff[j]);
                    if (!kin[j]) ksd[t][j] = 0;
                    if constexpr (KW == 4) {
                        const int4_t w = *reinterpret_cast<const int4_t *>(row + koff[j]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) kd[t][j][i] = (uint32_t)w[i];
                    } else {
                        const int2v_t w = *reinterpret_cast<const int2v_t *>(row + koff[j]);
                        kd[t][j][0] = (uint32_t)w[0];
                        kd[t][j][1] = (uint32_t)w[1];
                    }
                }
            }
        }
    };
    auto load_v = [&](int blk, const Ids &ids) {
        const int v = begin + 32 * blk;
        if constexpr (P16) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int vv = __builtin_amdgcn_readfirstlane(v + 16 * t), pid = __builtin_amdgcn_readfirstlane(ids.p[t]);
                const bool ok = vv < end && is_page(pid);
                const int kk = key_at(kr, vv), at = ok ? kk - key_page(a, kk) * a.page : 0, live = min(16, end - vv);
                const int64_t pg = ok ? pid : 0;
                const __amdgpu_buffer_rsrc_t r = make_rsrc(vbase + pg * a.v_ps + (int64_t)at * a.v_ts, ok ? (uint32_t)(live - 1) * a.v_ts + (uint32_t)a.D / 2 : 0u);
                const __amdgpu_buffer_rsrc_t rs = make_rsrc(vsbase + pg * a.vs_ps + (int64_t)at * a.s_ts, ok ? (uint32_t)live * a.s_ts : 0u);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int x = 0; x < VC; ++x) {
                        const uint32_t o = voff[x] == ATT_OOB ? ATT_OOB : voff[x] + i * a.v_ts, os = vsoff[x] == ATT_OOB ? ATT_OOB : vsoff[x] + i * a.s_ts;
                        vsd[4 * t + i][x] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rs, os, 0, 0);
                        if constexpr (VW == 8)
                            vd[4 * t + i][x] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, o, 0, 0);
                        else
                            vd[4 * t + i][x] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, o, 0, 0);
                    }
            }
        } else {
            const bool there = v + (lane & 31) < end && is_page(ids.p[0]);
            const int kk = key_at(kr, max(0, min(v + (lane & 31), end - 1))), at = kk - key_page(a, kk) * a.page, pg = there ? ids.p[0] : 0;
            const int64_t off = (int64_t)pg * a.v_ps + (int64_t)at * a.v_ts, soff = (int64_t)pg * a.vs_ps + (int64_t)at * a.s_ts;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int src = 16 * (e >> 2) + 4 * g + (e & 3);
                auto from = [&](int64_t x) {
                    const uint32_t lo = (uint32_t)__shfl((int)(uint32_t)x, src), hi = (uint32_t)__shfl((int)(x >> 32), src);
                    return (int64_t)(((uint64_t)hi << 32) | lo);
                };
                const uint8_t *row = vbase + from(off), *srow = vsbase + from(soff);
#pragma unroll
                for (int x = 0; x < VC; ++x) {
                    vsd[e][x] = *reinterpret_cast<const uint32_t *>(srow + vsoff[x]);
                    if (!vin[x]) vsd[e][x] = 0;
                    if constexpr (VW == 8)
                        vd[e][x] = *reinterpret_cast<const uint32_t *>(row + voff[x]);
                    else
                        vd[e][x] = *reinterpret_cast<const uint16_t *>(row + voff[x]);
                }
            }
        }
    };

    float m[QT], l[QT];
    float4_t o[QT][XT];
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        m[qt] = -INFINITY;
        l[qt] = 0.f;
#pragma unroll
        for (int x = 0; x < XT; ++x) o[qt][x] = float4_t{0.f, 0.f, 0.f, 0.f};
    }

    const int blocks = (max(0, end - begin) + 31) >> 5;
    if (wave < blocks) {
        Ids cur = ids_of(wave), nxt = ids_of(wave + NW);
        load_k(wave, cur);
        load_v(wave, cur);
        for (int blk = wave; blk < blocks; blk += NW) {
            const int v0 = begin + 32 * blk;
            float4_t s[QT][2];
#pragma unroll
            for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                for (int t = 0; t < 2; ++t) s[qt][t] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int jl = 0; jl < KL; ++jl) {
                    const Zero z = zero_of(ksd[t][jl], ksd[t][jl]);
#pragma unroll
                    for (int w = 0; w < KW; ++w) {
                        const int4_t kf = values8(kd[t][jl][w], z);
#pragma unroll
                        for (int qt = 0; qt < QT; ++qt) s[qt][t] = mfma_16(kf, q[qt][KW * jl + w], s[qt][t], f16_t());
                    }
                }
            // the next block's keys load under this block's softmax and second product
            load_k(blk + NW, nxt);

            // a half needs a look at its keys where not every row sees all of them
            int key0[2];
            bool masked = v0 + 32 > end;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                key0[t] = key_at(kr, v0 + 16 * t);
                masked = masked || key0[t] + 16 > all_hi || (key0[t] < all_lo && key0[t] + 16 > a.sinks);
                if constexpr (P16) masked = masked || !is_page(cur.p[t]);
            }
            if constexpr (!P16) masked = masked || __any(!is_page(cur.p[0]));
            if (masked) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = key0[t] + 4 * g + i;
                        const int pid = P16 ? cur.p[t] : __shfl(cur.p[0], 16 * t + 4 * g + i);     // (by all lanes)
                        const bool off = v0 + 16 * t + 4 * g + i >= end || !is_page(pid);
#pragma unroll
                        for (int qt = 0; qt < QT; ++qt)
                            if (off || key >= vhi[qt] || (key < vlo[qt] && key >= a.sinks)) s[qt][t][i] = -INFINITY;
                        // values that no row sees may hold anything: they meet p = 0 as zeros
                        if (off || key >= kr.hi || (key < kr.lo && key >= a.sinks)) {
#pragma unroll
                            for (int x = 0; x < VC; ++x) vsd[4 * t + i][x] = 0;
                        }
                    }
            }
            int4_t p[QT];
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) {
                float x[8], mx = -INFINITY;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] = s[qt][e >> 2][e & 3] * sl[qt];
                    mx = fmaxf(mx, x[e]);
                }
                mx = fmaxf(mx, __shfl_xor(mx, 16));
                mx = fmaxf(mx, __shfl_xor(mx, 32));
                const float mn = fmaxf(m[qt], mx), ms = mn == -INFINITY ? 0.f : mn;
                if (__any(mn > m[qt])) {
                    const float al = __builtin_amdgcn_exp2f(m[qt] - ms);
                    l[qt] *= al;
#pragma unroll
                    for (int xx = 0; xx < XT; ++xx) o[qt][xx] *= al;
                    m[qt] = mn;
                }
                const float base = ms - A4_TOP;
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] = __builtin_amdgcn_exp2f(x[e] - base);
                    sum += x[e];
                }
                l[qt] += sum;
                p[qt] = int4_t{pack2(x[0], x[1], f16_t()), pack2(x[2], x[3], f16_t()), pack2(x[4], x[5], f16_t()), pack2(x[6], x[7], f16_t())};
            }
#pragma unroll
            for (int x = 0; x < VC; ++x) {
                Zero z[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) z[y] = zero_of(vsd[2 * y][x], vsd[2 * y + 1][x]);
#pragma unroll
                for (int h = 0; h < VW / 4; ++h) {
                    // four elements of two keys a dword
                    uint32_t w[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) w[y] = __builtin_amdgcn_perm(vd[2 * y + 1][x], vd[2 * y][x], h ? 0x07060302u : 0x05040100u);
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        int4_t vf;
#pragma unroll
                        for (int y = 0; y < 4; ++y) vf[y] = n & 1 ? value2<true>(w[y] >> (n & 2 ? 8 : 0), z[y]) : value2<false>(w[y] >> (n & 2 ? 8 : 0), z[y]);
#pragma unroll
                        for (int qt = 0; qt < QT; ++qt) o[qt][VW * x + 4 * h + n] = mfma_16(vf, p[qt], o[qt][VW * x + 4 * h + n], f16_t());
                    }
                }
            }
            load_v(blk + NW, nxt);
            cur = nxt;
            nxt = ids_of(blk + 2 * NW);
        }
    }

    // join the waves
    float *ml = att_lds + NW * nrow * LD;      // [wave][row][m, l]
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        l[qt] += __shfl_xor(l[qt], 16);
        l[qt] += __shfl_xor(l[qt], 32);
        const int row = 16 * qt + c;
        if (row < nrow) {
            float *dst = att_lds + (wave * nrow + row) * LD;
#pragma unroll
            for (int x = 0; x < XT; x += 4)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<float4_t *>(dst + 16 * VW * (x / VW) + VW * (4 * g + i) + x % VW) =
                        float4_t{o[qt][x][i], o[qt][x + 1][i], o[qt][x + 2][i], o[qt][x + 3][i]};
            if (g == 0) {
                ml[(wave * nrow + row) * 2] = m[qt];
                ml[(wave * nrow + row) * 2 + 1] = l[qt];
            }
        }
    }
    __syncthreads();
    const int d4 = a.D >> 2;
    for (int it = threadIdx.x; it < nrow * d4; it += 64 * NW) {
        const int row = it / d4, d = 4 * (it - row * d4);
        float mm = -INFINITY;
#pragma unroll
        for (int w = 0; w < NW; ++w) mm = fmaxf(mm, ml[(w * nrow + row) * 2]);
        const float ms = mm == -INFINITY ? 0.f : mm;
        float tot = 0.f;
        float4_t sum = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float f = __builtin_amdgcn_exp2f(ml[(w * nrow + row) * 2] - ms);
            tot += f * ml[(w * nrow + row) * 2 + 1];
            sum += f * *reinterpret_cast<const float4_t *>(att_lds + (w * nrow + row) * LD + d);
        }
        const int r = rb * a.rows + row, i = r / a.g, hq = hk * a.g + (r - i * a.g);
        const int64_t t = kr.t0 + i;
        // no sum: no key, or scores of -inf by overflow (of a split: the join looks)
        const bool none = tot == 0.f && (a.splits > 1 || !row_sees(a, b, kr, i));
        const float inv = 1.f / (tot > 0.f ? tot : NAN);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = none ? 0.f : sum[e] * inv;
        const float lse2 = none ? -INFINITY : mm - A4_TOP + __builtin_amdgcn_logf(tot > 0.f ? tot : NAN);
        if (a.splits == 1) {
            *reinterpret_cast<int2v_t *>((char *)a.out + t * a.o_ts + (int64_t)hq * a.o_hs + 2 * d) =
                int2v_t{pack2(sum[0], sum[1], tag), pack2(sum[2], sum[3], tag)};
            if (a.lse && d == 0) a.lse[t * a.Hq + hq] = lse2 * ATT_LN2;
        } else {
            const int64_t at = (t * a.Hq + hq) * a.splits + split;
            *reinterpret_cast<float4_t *>(a.part + at * a.D + d) = sum;
            if (d == 0) a.part[(int64_t)a.T * a.Hq * a.splits * a.D + at] = lse2;
        }
    }
}

// ---------------------------------------------------------------------------
// Many query rows for each key head (prompts, chunks): as attend_tiles_kernel, a
// workgroup of NW waves takes 32 NW rows of one (sequence, key head) and one split of
// the places; the waves share tiles of keys and values in LDS as f16, which the threads
// that stage them make out of the codes: once for all rows.
// Keys stand in LDS in codes' order within each 8 elements (q's rows do too), values in
// their own.
// ---------------------------------------------------------------------------
__host__ __device__ constexpr int tiles4_keys(int D) { return D <= 128 ? 64 : 32; }
__host__ __device__ constexpr int tiles4_waves(int D) { return D <= 128 ? 8 : 4; }
constexpr float A4_LAZY = 4.f;         // a maximum may be exceeded by this much (base 2)

// 8 codes of a dword as f16, in their own order: byte b's two codes stand at bits 0 and 20
__device__ __forceinline__ int4_t values8_in_order(uint32_t w, uint32_t sc)
{
    const f16_t s = as_half((uint16_t)sc), z = as_half((uint16_t)(sc >> 16));
    const half2_t off = half2_t{(f16_t)-1024.f - z, (f16_t)-64.f - z}, part = half2_t{(f16_t)1.f, (f16_t)0.0625f}, ss = half2_t{s, s};
    int4_t r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t two = __builtin_amdgcn_perm(w, w, i == 0 ? 0x0c000c00u : i == 1 ? 0x0c010c01u : i == 2 ? 0x0c020c02u : 0x0c030c03u);
        r[i] = (int)as_u32(__builtin_elementwise_fma(as_half2(qmm_and_or(two, 0x00f0000fu, 0x64006400u)), part, off) * ss);
    }
    return r;
}

template <typename S, int DC, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(DC <= 128 ? 2 : 1, DC <= 128 ? 2 : 1))) void attend4_tiles_kernel(const Attend4Args a)
{
    constexpr int DP = DC == 96 ? 128 : DC;              // pitch of a row in LDS; DC elements of it are computed
    constexpr int KB = tiles4_keys(DP), KT = KB / 32;    // keys of a tile, halves of 32 of them
    constexpr int CH = DP / 8;                           // 16-byte chunks of a row in LDS
    constexpr int LN = KB * CH / (64 * NW);              // chunks of K (and of V) a thread stages
    constexpr int QJ = DC / 16, XT = DC / 32;
    constexpr int TILE = KB * DP * 2;                    // bytes
    constexpr float TOP = A4_TOP - A4_LAZY;
    auto swizzle_k = [](int row) { return CH == 8 ? (row >> 1) & 7 : row & 15; };
    auto swizzle_v = [](int row) { return CH == 8 ? 4 * ((row >> 1) & 1) : 4 * (row & 3); };
    extern __shared__ __attribute__((aligned(16))) uint8_t att_tiles[];   // K [2][TILE], V [2][TILE]
    typedef __attribute__((address_space(3))) short4v_t lds4_t;

    int id = blockIdx.x;
    const int groups = a.B * a.Hkv;
    const int bh = id % groups;                          // sequence and head fastest: one head's blocks share an L2
    id /= groups;
    const int split = id % a.splits, rb = a.rblocks - 1 - id / a.splits;   // the longest blocks first
    const int b = bh / a.Hkv, hk = bh - b * a.Hkv;

    const Range4 kr = range4(a, b, rb);
    const int nrow = min(32 * NW, kr.n * a.g - rb * a.rows);
    if (nrow <= 0) return;
    const int begin = split * a.chunk, end = min(kr.len, begin + a.chunk);
    if (begin >= end && split > 0) return;

    const int tid = threadIdx.x, lane = tid & 63, wave = wave_id(), c = lane & 31, h = lane >> 5;
    const S tag = (S)0.f;

    // this lane's row
    const int r = rb * a.rows + 32 * wave + c, i = r / a.g, hq = hk * a.g + (r - i * a.g);
    const bool live = 32 * wave + c < nrow;
    const int vhi = live ? kr.L - kr.n + i + 1 : 0, vlo = a.window > 0 ? vhi - a.window : 0;
    int4_t q[QJ];
    float sl = a.scale * ATT_LOG2E;
    {
        const char *row = (const char *)a.q + (int64_t)(kr.t0 + (live ? i : 0)) * a.q_ts + (int64_t)(live ? hq : 0) * a.q_hs;
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < QJ; ++j) {
            const int d = 16 * j + 8 * h;
            q[j] = *reinterpret_cast<const int4_t *>(row + (d < a.D ? 2 * d : 0));
            if (!live || d >= a.D) q[j] = int4_t{0, 0, 0, 0};
            if constexpr (!__is_same(S, f16_t)) top = fmaxf(top, largest(q[j], tag));
        }
        if constexpr (!__is_same(S, f16_t)) {
            const int up = rise_of(fmaxf(top, __shfl_xor(top, 32)));
#pragma unroll
            for (int j = 0; j < QJ; ++j) q[j] = to_f16(q[j], up);
            sl = ldexpf(sl, -up);
        }
        sl = above_zero(sl);
#pragma unroll
        for (int j = 0; j < QJ; ++j) q[j] = code_order(q[j]);
    }
    // keys that some row of the wave sees, and keys that all of them see
    const int wr0 = rb * a.rows + 32 * wave, wr1 = min(wr0 + 31, rb * a.rows + nrow - 1);
    const bool wlive = 32 * wave < nrow;
    const int whi = wlive ? kr.L - kr.n + wr1 / a.g + 1 : 0, wall_hi = wlive ? kr.L - kr.n + wr0 / a.g + 1 : 0;
    const int wlo = a.window > 0 ? wall_hi - a.window : 0, wall_lo = a.window > 0 ? whi - a.window : 0;

    const uint8_t *kbase = a.k + (int64_t)hk * a.k_hs, *vbase = a.v + (int64_t)hk * a.v_hs;
    const uint8_t *ksbase = (const uint8_t *)a.ks + (int64_t)hk * a.ks_hs, *vsbase = (const uint8_t *)a.vs + (int64_t)hk * a.vs_hs;
    const int32_t *table = a.table + (int64_t)b * a.table_s;

    // Where the rows stand: every NW tiles each wave looks up one of the NW tiles after the
    // current ones, lane l the place number l of it, and leaves where its codes and scales are
    // in both caches in LDS (2 NW slots), with two masks: keys that some row may see, keys
    // on bad pages.  A place past the end takes the last one's and a bad page id page
    // 0's: in bounds, and hidden.
    constexpr int SLOTS = 2 * NW;
    int4_t *places = reinterpret_cast<int4_t *>(att_tiles + 4 * TILE);       // [SLOTS][KB][2]: codes of K low, high, of V; scales likewise
    int4_t *masks = places + 2 * SLOTS * KB;                                 // [SLOTS]: seen low, high, bad low, high
    auto key_of = [&](int tile) { return key_at(kr, max(0, min(begin + KB * tile + (lane & (KB - 1)), end - 1))); };
    auto ids_of = [&](int tile) { return table[key_page(a, key_of(tile))]; };
    auto two = [](int64_t x, int64_t y) { return int4_t{(int)(uint32_t)x, (int)(x >> 32), (int)(uint32_t)y, (int)(y >> 32)}; };
    auto look_up = [&](int tile, int pid) {
        const int v = begin + KB * tile + (lane & (KB - 1)), key = key_of(tile), at = key - key_page(a, key) * a.page;
        const bool ok = (uint32_t)pid < (uint32_t)a.pages;
        const uint64_t seen = __ballot(ok && v < end && key < kr.hi && (key >= kr.lo || key < kr.sk)), bad = __ballot(!ok);
        const int64_t pg = ok ? pid : 0;
        const int slot = tile % SLOTS;
        if (lane < KB) {
            places[2 * (slot * KB + lane)] = two(pg * a.k_ps + (int64_t)at * a.k_ts, pg * a.v_ps + (int64_t)at * a.v_ts);
            places[2 * (slot * KB + lane) + 1] = two(pg * a.ks_ps + (int64_t)at * a.s_ts, pg * a.vs_ps + (int64_t)at * a.s_ts);
        }
        if (lane == 0) masks[slot] = int4_t{(int)(uint32_t)seen, (int)(uint32_t)(seen >> 32), (int)(uint32_t)bad, (int)(uint32_t)(bad >> 32)};
    };
    const int srow = tid / CH, sp = tid % CH;             // this thread stages rows srow + SSTEP n, chunk sp
    constexpr int SSTEP = 64 * NW / CH;
    const int in_row = 8 * sp < a.D ? 4 * sp : 0, in_scales = 8 * sp < a.D ? 4 * ((8 * sp) >> a.lg_G) : 0;
    uint32_t kst[LN], vst[LN], kss[LN], vss[LN];
    uint64_t vlive = 0, hidden = 0;                       // the masks of the staged tile
    auto uniform64 = [](int lo, int hi) {
        return ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane(hi) << 32) | (uint32_t)__builtin_amdgcn_readfirstlane(lo);
    };
    auto off64 = [](int lo, int hi) { return (int64_t)(((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo); };
    auto load_tile = [&](int tile) {
        const int slot = tile % SLOTS;
        const int4_t mk = masks[slot];
#pragma unroll
        for (int n = 0; n < LN; ++n) {
            const int4_t at = places[2 * (slot * KB + srow + SSTEP * n)], as = places[2 * (slot * KB + srow + SSTEP * n) + 1];
            kst[n] = *reinterpret_cast<const uint32_t *>(kbase + off64(at[0], at[1]) + in_row);
            vst[n] = *reinterpret_cast<const uint32_t *>(vbase + off64(at[2], at[3]) + in_row);
            kss[n] = *reinterpret_cast<const uint32_t *>(ksbase + off64(as[0], as[1]) + in_scales);
            vss[n] = *reinterpret_cast<const uint32_t *>(vsbase + off64(as[2], as[3]) + in_scales);
        }
        vlive = uniform64(mk[0], mk[1]);
        hidden = uniform64(mk[2], mk[3]);
    };
    auto store_tile = [&](int buf) {
        if (~vlive) {     // what no row sees may hold anything: it meets p = 0 as zeros
#pragma unroll
            for (int n = 0; n < LN; ++n) vss[n] = (vlive >> (srow + SSTEP * n)) & 1 ? vss[n] : 0;
        }
        const bool in = 8 * sp < a.D;
#pragma unroll
        for (int n = 0; n < LN; ++n) {
            const int row = srow + SSTEP * n;
            const uint32_t ks = in ? kss[n] : 0;          // (elements past D meet zeros of q: finite will do)
            *reinterpret_cast<int4_t *>(att_tiles + buf * TILE + row * DP * 2 + 16 * (sp ^ swizzle_k(row))) = values8(kst[n], zero_of(ks, ks));
            *reinterpret_cast<int4_t *>(att_tiles + (2 + buf) * TILE + row * DP * 2 + 16 * (sp ^ swizzle_v(row))) = values8_in_order(vst[n], vss[n]);
        }
    };

    // LDS addresses of this lane's operands: K row c, chunk 2 j + h; V block: rows 4 h + lane % 16 / 4,
    // columns 16 (lane / 16 % 2) + 4 (lane % 4) of the 32 of step x.  (The swizzles change 4 bits of the
    // chunk at most: the other steps lie 256 bytes apart.)
    constexpr int KA = QJ < 8 ? QJ : 8, VA = XT < 4 ? XT : 4;
    uint32_t ka[KA], va[VA];
#pragma unroll
    for (int j = 0; j < KA; ++j) ka[j] = (uint32_t)(c * DP * 2 + 16 * ((2 * j + h) ^ swizzle_k(c)));
    {
        const int l16 = lane & 15, row = 4 * h + (l16 >> 2);
#pragma unroll
        for (int x = 0; x < VA; ++x) {
            const int chunk = (4 * x + 2 * ((lane >> 4) & 1) + ((l16 & 3) >> 1)) ^ swizzle_v(row);
            va[x] = (uint32_t)(2 * TILE + row * DP * 2 + 16 * chunk + 8 * (l16 & 1));
        }
    }

    float m = -INFINITY, l = 0.f;
    float16v_t o[XT];
#pragma unroll
    for (int x = 0; x < XT; ++x)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[x][e] = 0.f;

    const int tiles = (max(0, end - begin) + KB - 1) / KB;
    look_up(wave, ids_of(wave));
    int pid = ids_of(NW + wave);
    __syncthreads();
    load_tile(0);
    uint64_t bad = hidden;
    store_tile(0);
    __syncthreads();
    for (int tile = 0; tile < tiles; ++tile) {
        const int buf = tile & 1, v0 = begin + KB * tile, key0 = key_at(kr, v0);
        load_tile(tile + 1);
        if (tile % NW == 0) {
            look_up(tile + NW + wave, pid);
            pid = ids_of(tile + 2 * NW + wave);
        }
        if (key0 < whi && (key0 + KB > wlo || key0 < kr.sk)) {
            const uint8_t *kl = att_tiles + buf * TILE;
            // operands are read from LDS KA steps ahead of the products that take them
            auto read_k = [&](int n) {     // step n of KT QJ: tile n / QJ, step n % QJ
                const int t = n / QJ, j = n % QJ;
                return *reinterpret_cast<const int4_t *>(kl + ka[j % KA] + 256 * (j / KA) + t * 32 * DP * 2);
            };
            auto read_v = [&](int n) {     // step n of 2 KT XT: keys 16 (n / XT), columns 32 (n % XT)
                const int u = n / XT, x = n % XT;
                const uint32_t at = va[x % VA] + buf * TILE + 256 * (x / VA) + u * 16 * DP * 2;
                const int2v_t w0 = __builtin_bit_cast(int2v_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4_t *)(att_tiles + at)));
                const int2v_t w1 = __builtin_bit_cast(int2v_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4_t *)(att_tiles + at + 8 * DP * 2)));
                return int4_t{w0[0], w0[1], w1[0], w1[1]};
            };
            float16v_t s[KT];
            int4_t kf[KA], vf[VA];
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int n = 0; n < KA; ++n) kf[n] = read_k(n);
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int e = 0; e < 16; ++e) s[t][e] = 0.f;
#pragma unroll
            for (int n = 0; n < KT * QJ; ++n) {
                s[n / QJ] = mfma_32(kf[n % KA], q[n % QJ], s[n / QJ], f16_t());
                if (n + KA < KT * QJ)
                    kf[n % KA] = read_k(n + KA);
                else if (n + KA - KT * QJ < VA)
                    vf[n + KA - KT * QJ] = read_v(n + KA - KT * QJ);
            }
            __builtin_amdgcn_sched_group_barrier(0x100, KA, 0);
#pragma unroll
            for (int n = 0; n < KT * QJ; ++n) {
                __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
                if (n + KA < KT * QJ)
                    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
                else if (n + KA - KT * QJ < VA)
                    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (v0 + KB > end || key0 + KB > wall_hi || (key0 < wall_lo && key0 + KB > kr.sk) || bad) {
                // element e of tile t is key key0 + 4 h + kt, kt a constant (v0 + KB > end with the last places alone: key >= vhi there)
                const int to = min(vhi, key0 + end - v0) - key0 - 4 * h, from = vlo - key0 - 4 * h, sinks = kr.sk - key0 - 4 * h;
                const uint64_t hide = bad >> (4 * h);
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int kt = 32 * t + (e & 3) + 8 * (e >> 2);
                        const bool off = kt >= to || (kt < from && kt >= sinks) || ((uint32_t)(hide >> (32 * t)) & (1u << (kt & 31)));
                        s[t][e] = off ? -INFINITY : s[t][e];
                    }
            }
            float mx = s[0][0];
#pragma unroll
            for (int e = 1; e < 16 * KT; ++e) mx = fmaxf(mx, s[e >> 4][e & 15]);
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            mx *= sl;
            if (__any(mx > m + A4_LAZY)) {               // also the first finite maximum: m is -inf
                const float mn = fmaxf(m, mx), al = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.f : mn));
                l *= al;
#pragma unroll
                for (int x = 0; x < XT; ++x) o[x] *= al;
                m = mn;
            }
            const float base = (m == -INFINITY ? 0.f : m) - TOP;
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 16 * KT; ++e) {
                const float p = __builtin_amdgcn_exp2f(fmaf(s[e >> 4][e & 15], sl, -base));
                sum += p;
                s[e >> 4][e & 15] = p;
            }
            l += sum;
#pragma unroll
            for (int u = 0; u < 2 * KT; ++u) {
                int4_t p;
#pragma unroll
                for (int e = 0; e < 4; ++e) p[e] = pack2(s[u >> 1][8 * (u & 1) + 2 * e], s[u >> 1][8 * (u & 1) + 2 * e + 1], f16_t());
#pragma unroll
                for (int x = 0; x < XT; ++x) {
                    const int n = u * XT + x;
                    o[x] = mfma_32(vf[n % VA], p, o[x], f16_t());
                    if (n + VA < 2 * KT * XT) vf[n % VA] = read_v(n + VA);
                }
            }
        }
        bad = hidden;
        store_tile(buf ^ 1);
        __syncthreads();
    }

    l += __shfl_xor(l, 32);
    if (!live) return;
    const bool none = l == 0.f && (a.splits > 1 || !row_sees(a, b, kr, i));
    const float tot = l > 0.f ? l : NAN, inv = 1.f / tot;
    const float lse2 = none ? -INFINITY : m - TOP + __builtin_amdgcn_logf(tot);
    const int64_t t = kr.t0 + i, at = (t * a.Hq + hq) * a.splits + split;
    char *out = (char *)a.out + t * a.o_ts + (int64_t)hq * a.o_hs;
#pragma unroll
    for (int x = 0; x < XT; ++x)
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
            const int d = 32 * x + 2 * e + 4 * h;
            if (d >= a.D) continue;
            float4_t y;
#pragma unroll
            for (int k = 0; k < 4; ++k) y[k] = none ? 0.f : o[x][e + k] * inv;
            if (a.splits == 1)
                *reinterpret_cast<int2v_t *>(out + 2 * d) = int2v_t{pack2(y[0], y[1], tag), pack2(y[2], y[3], tag)};
            else
                *reinterpret_cast<float4_t *>(a.part + at * a.D + d) = y;
        }
    if (h == 0) {
        if (a.splits > 1)
            a.part[(int64_t)a.T * a.Hq * a.splits * a.D + at] = lse2;
        else if (a.lse)
            a.lse[t * a.Hq + hq] = lse2 * ATT_LN2;
    }
}

// Joins the splits: as attend_join_kernel.
template <typename S, int DP, int JW>
__global__ __launch_bounds__(256) void attend4_join_kernel(const Attend4Args a)
{
    constexpr int LN = DP / 4, SW = 64 / LN;        // lanes of a split, splits of a wave
    constexpr int RG = 4 / JW;                      // rows of the workgroup
    __shared__ __attribute__((aligned(16))) float sums[4][DP];
    __shared__ float tots[4];
    const int per = (int)(((int64_t)a.max_q * a.Hq + RG - 1) / RG);
    const int b = blockIdx.x / per, wave = wave_id(), part_wave = wave % JW, lane = threadIdx.x & 63;
    const int r = (blockIdx.x - b * per) * RG + wave / JW, i = r / a.Hq, hq = r - i * a.Hq;
    const int rb = (min(i, a.max_q - 1) * a.g + hq % a.g) / a.rows;
    const Range4 kr = range4(a, b, rb);
    const bool live = i < a.max_q && i < kr.n;
    if (JW == 4 && !live) return;                    // the whole workgroup
    const int splits = live ? max(1, (kr.len + a.chunk - 1) / a.chunk) : 0;
    const int64_t row = live ? (int64_t)(kr.t0 + i) * a.Hq + hq : 0;
    const float *lses = a.part + (int64_t)a.T * a.Hq * a.splits * a.D + row * a.splits;
    float mm = -INFINITY;
    for (int s = lane; s < splits; s += 64) mm = fmaxf(mm, lses[s]);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) mm = fmaxf(mm, __shfl_xor(mm, x));
    const float ms = mm == -INFINITY ? 0.f : mm;
    const int d = 4 * (lane % LN);
    const float *part = a.part + row * a.splits * a.D + (d < a.D ? d : 0);
    float4_t sum = float4_t{0.f, 0.f, 0.f, 0.f};
    float tot = 0.f;
#pragma unroll 4
    for (int s = part_wave * SW + lane / LN; s < splits; s += JW * SW) {
        const float f = __builtin_amdgcn_exp2f(lses[s] - ms);
        tot += f;
        sum += f * *reinterpret_cast<const float4_t *>(part + (int64_t)s * a.D);
    }
#pragma unroll
    for (int x = LN; x < 64; x <<= 1) {
        tot += __shfl_xor(tot, x);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] += __shfl_xor(sum[e], x);
    }
    if constexpr (JW > 1) {
        if (lane < LN) *reinterpret_cast<float4_t *>(&sums[wave][d]) = sum;
        if (lane == 0) tots[wave] = tot;
        __syncthreads();
        if (part_wave != 0) return;
        tot = 0.f;
        sum = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < JW; ++w) {
            tot += tots[wave + w];
            sum += *reinterpret_cast<const float4_t *>(&sums[wave + w][d]);
        }
    }
    if (!live) return;
    const bool none = tot == 0.f && !row_sees(a, b, kr, i);
    tot = tot > 0.f ? tot : NAN;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = none ? 0.f : sum[e] * (1.f / tot);
    if (lane < LN && d < a.D)
        *reinterpret_cast<int2v_t *>((char *)a.out + (int64_t)(kr.t0 + i) * a.o_ts + (int64_t)hq * a.o_hs + 2 * d) =
            int2v_t{pack2(sum[0], sum[1], (S)0.f), pack2(sum[2], sum[3], (S)0.f)};
    if (a.lse && lane == 0) a.lse[row] = none ? -INFINITY : (mm + __builtin_amdgcn_logf(tot)) * ATT_LN2;
}

constexpr int ROWS4_NW = 4;     // waves of a rows workgroup

int64_t plan_attend4(Attend4Args &a)
{
    int lg = 0;                // key / page by one multiplication, as in plan_attend
    while ((int64_t(1) << lg) < a.page) ++lg;
    a.page_mul = (uint32_t)((uint64_t(1) << (31 + lg)) / (uint64_t)a.page + 1);
    a.page_sh = 31 + lg;

    const int64_t rows = (int64_t)a.max_q * a.g;
    const bool tiles = rows > 32;
    a.rows = tiles ? 32 * tiles4_waves(a.D) : rows <= 16 || a.D > 128 ? 16 : 32;
    a.rblocks = (int)((rows + a.rows - 1) / a.rows);
    a.unit = tiles ? tiles4_keys(a.D) : 16;
    int64_t span = a.max_kv;
    if (a.window > 0)
        span = std::min(span, (int64_t)a.window + (a.rows + a.g - 1) / a.g + (std::min<int64_t>(a.sinks, a.max_kv) + a.unit - 1) / a.unit * a.unit);
    span += 15;
    const int64_t groups = (int64_t)a.B * a.Hkv * a.rblocks;
    int64_t splits, unit;
    if (tiles) {
        unit = 128;
        splits = std::max(std::min(256 / groups, span / 320), std::min((512 + groups - 1) / groups, span / 2048));
    } else {
        unit = 32 * ROWS4_NW;
        const int64_t bytes = (span - 15) * (a.D + 8 * (a.D >> a.lg_G)), kb = 1024;
        splits = std::max(std::min(256 / groups, (bytes + 32 * kb - 1) / (32 * kb)),
                          std::max<int64_t>(1, std::min((768 + groups - 1) / groups, (bytes + 64 * kb - 1) / (64 * kb))));
        splits *= (std::max<int64_t>(1, bytes / splits) + 1152 * kb - 1) / (1152 * kb);
        if (bytes <= std::max<int64_t>(112, std::min<int64_t>(512, 2 * groups)) * kb) splits = 1;
    }
    splits = std::max<int64_t>(1, splits);
    a.chunk = (int)(((span + splits - 1) / splits + unit - 1) / unit * unit);
    a.splits = (int)((span + a.chunk - 1) / a.chunk);
    return a.splits > 1 ? (int64_t)a.T * a.Hq * a.splits * (a.D + 1) * 4 : 0;
}

template <typename K>
static hipError_t allow_lds(K *kernel, size_t bytes)
{
    return bytes <= 64 * 1024 ? hipSuccess
                              : hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
}

template <typename S, int DC>
static hipError_t tiles4_go(const Attend4Args &a, hipStream_t st)
{
    constexpr int DP = DC == 96 ? 128 : DC, NW = tiles4_waves(DP), KB = tiles4_keys(DP);
    const size_t lds = (size_t)4 * KB * DP * 2 + 2 * NW * (2 * KB + 1) * 16;   // tiles, places, masks
    const hipError_t e = allow_lds(&attend4_tiles_kernel<S, DC, NW>, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((attend4_tiles_kernel<S, DC, NW>), dim3((unsigned)((int64_t)a.B * a.rblocks * a.Hkv * a.splits)), dim3(64 * NW), lds, st, a);
    return hipGetLastError();
}

template <typename S, int DP, bool P16, int QT>
static hipError_t rows4_go(const Attend4Args &a, hipStream_t st)
{
    constexpr int NW = ROWS4_NW;
    const int nrow = (int)std::min<int64_t>(16 * QT, (int64_t)a.max_q * a.g);
    const size_t lds = (size_t)NW * nrow * (DP + 6) * 4;
    const hipError_t e = allow_lds(&attend4_rows_kernel<S, DP, P16, QT, NW>, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((attend4_rows_kernel<S, DP, P16, QT, NW>), dim3((unsigned)((int64_t)a.B * a.rblocks * a.Hkv * a.splits)), dim3(64 * NW), lds, st, a);
    return hipGetLastError();
}

template <typename S, int DP, bool P16>
static hipError_t rows4_pick(const Attend4Args &a, hipStream_t st)
{
    if constexpr (DP <= 128) {
        if (a.rows == 32) return rows4_go<S, DP, P16, 2>(a, st);
    }
    return rows4_go<S, DP, P16, 1>(a, st);
}

// A wave a row where the splits are few, the workgroup's four where a single wave would
// read them in more than four rounds.
static int join4_waves(const Attend4Args &a) { return a.splits <= 4 * (256 / (a.D <= 64 ? 64 : a.D <= 128 ? 128 : 256)) ? 1 : 4; }
static int64_t join4_blocks(const Attend4Args &a)     // for each sequence
{
    const int64_t rows = (int64_t)a.max_q * a.Hq;
    return join4_waves(a) == 1 ? (rows + 3) / 4 : rows;
}
template <typename S, int DP>
static hipError_t join4_go(const Attend4Args &a, hipStream_t st)
{
    const dim3 grid((unsigned)(join4_blocks(a) * a.B));
    if (join4_waves(a) == 1)
        hipLaunchKernelGGL((attend4_join_kernel<S, DP, 1>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((attend4_join_kernel<S, DP, 4>), grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

template <typename S>
static hipError_t attend4_type(const Attend4Args &a, hipStream_t st)
{
    hipError_t e;
    if (a.rows > 32)
        e = a.D <= 64 ? tiles4_go<S, 64>(a, st) : a.D <= 96 ? tiles4_go<S, 96>(a, st) : a.D <= 128 ? tiles4_go<S, 128>(a, st) : tiles4_go<S, 256>(a, st);
    else if (a.D <= 64)
        e = a.halves ? rows4_pick<S, 64, true>(a, st) : rows4_pick<S, 64, false>(a, st);
    else if (a.D <= 128)
        e = a.halves ? rows4_pick<S, 128, true>(a, st) : rows4_pick<S, 128, false>(a, st);
    else
        e = a.halves ? rows4_pick<S, 256, true>(a, st) : rows4_pick<S, 256, false>(a, st);
    if (e != hipSuccess || a.splits == 1) return e;
    if (a.D <= 64) return join4_go<S, 64>(a, st);
    if (a.D <= 128) return join4_go<S, 128>(a, st);
    return join4_go<S, 256>(a, st);
}

// A launch takes fewer than 2^32 threads.  Both launches of a call are looked at before
// the first: a call is made whole or not at all.
static bool attend4_fits(const Attend4Args &a)
{
    const int64_t most = (int64_t(1) << 32) - 1, groups = (int64_t)a.B * a.Hkv;
    const int64_t threads = 64 * (a.rows > 32 ? tiles4_waves(a.D) : ROWS4_NW);
    if (groups > most || a.rblocks * groups > most / threads / a.splits) return false;
    return a.splits == 1 || join4_blocks(a) <= most / 256 / a.B;
}

hipError_t launch_attend4(const Attend4Args &a, bool bf16, hipStream_t st)
{
    if (!attend4_fits(a)) return hipErrorNotSupported;
    return bf16 ? attend4_type<bf16_t>(a, st) : attend4_type<f16_t>(a, st);
}

}  // namespace qmm
