// attend.hip -- attention of new tokens over a paged KV cache.
//
//     o_i = sum_j p_ij v_j,   p_ij = exp(x_ij - max_j x_ij) / sum_j exp(..),   x_ij = scale q_i . k_j
//
// over the keys j that row i sees: j <= L - n + i (L keys in the sequence, n
// of them new), and j > L - n + i - window where there is a window.  A row
// that sees no key gives zeros and a log sum of -inf.  A row whose scores are
// all NaN, or all -inf by overflow, leaves m at -inf too: whether it sees a key is
// asked of the table then, and if it does its output and log sum are NaN.
//
// One pass over the keys with a running maximum m and sum l (fp32), in base 2:
// x is scaled by log2(e), so p is one v_exp_f32; O and l are scaled by
// 2^(m_old - m_new) where a maximum rises.
#include <algorithm>
#include <math.h>

#include "launch.hpp"
#include "qmm_device.hpp"
#include "elem.hpp"

namespace qmm {

typedef __bf16 bf8x_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf2x_t __attribute__((ext_vector_type(2)));
typedef int int2v_t __attribute__((ext_vector_type(2)));

constexpr uint32_t ATT_OOB = 0x80000000u;
constexpr float ATT_LOG2E = 1.44269504088896340736f, ATT_LN2 = 0.69314718055994530942f;

__device__ __forceinline__ float4_t mfma_16(int4_t a, int4_t b, float4_t c, _Float16)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
}
__device__ __forceinline__ float4_t mfma_16(int4_t a, int4_t b, float4_t c, bf16_t)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8x_t, a), __builtin_bit_cast(bf8x_t, b), c, 0, 0, 0);
}

// two fp32 -> a dword of two elements, each rounded to nearest even
__device__ __forceinline__ int pack2(float x, float y, _Float16) { return __builtin_bit_cast(int, half2_t{(_Float16)x, (_Float16)y}); }
__device__ __forceinline__ int pack2(float x, float y, bf16_t) { return __builtin_bit_cast(int, bf2x_t{(bf16_t)x, (bf16_t)y}); }

// Probabilities meet the values in S.  fp16 is in full down to 2^-14 and ends at 2^-25:
// with a row's largest at 1, keys more than 10 below it in the exponent would lose bits and
// keys more than 17 below it would count in l alone, and beside a largest key without a
// value a long row of them is all there is.  In fp16 p and l are therefore scaled by 2^15:
// in full down to 2^-29 of the largest, off by 2^-40 of it beyond (2000 keys 15 below one
// of value 0: 2.6 % off without).  bf16 has fp32's exponents.  No time: it is part of the
// maximum that is subtracted.
template <typename S> constexpr float ATT_TOP = 0.f;
template <> constexpr float ATT_TOP<_Float16> = 15.f;

// two e4m3 (low or high half of a dword) -> two elements; exact in both types
template <bool HI> __device__ __forceinline__ int widen(int w, _Float16)
{
    return __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((uint32_t)w, 1.0f, HI));
}
template <bool HI> __device__ __forceinline__ int widen(int w, bf16_t)
{
    return __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((uint32_t)w, 1.0f, HI));
}

// The keys of a block of rows: [lo, hi) is what any of its rows sees; start is
// lo brought down to a multiple of 16.
struct KeyRange {
    int t0, n, L, lo, hi, start;
};
__device__ __forceinline__ KeyRange key_range(const AttendArgs &a, int b, int rb)
{
    KeyRange r;
    int t0 = a.cu_q[b], n = a.cu_q[b + 1] - t0;
    if (t0 < 0 || n < 0 || t0 + (int64_t)n > a.T) n = 0;
    n = min(n, a.max_q);
    r.t0 = t0;
    r.n = n;
    r.L = (int)min((int64_t)max(a.kv_lens[b], 0), min((int64_t)a.width * a.page, (int64_t)a.max_kv));
    const int first = rb * a.rows / a.g, last = (min((rb + 1) * a.rows, n * a.g) - 1) / a.g;
    r.hi = max(0, min(r.L, r.L - n + last + 1));
    r.lo = a.window > 0 ? max(0, r.L - n + first - a.window + 1) : 0;
    r.start = r.lo & ~15;
    return r;
}

__device__ __forceinline__ int key_page(const AttendArgs &a, int key)
{
    return (int)(((uint64_t)(uint32_t)key * a.page_mul) >> a.page_sh);
}

// Whether one of the keys [lo, hi) of sequence b stands on a page of the cache.
// Asked of rows without a sum alone.
__device__ __forceinline__ bool sees_key(const AttendArgs &a, int b, int64_t lo, int64_t hi)
{
    for (int64_t key = lo > 0 ? lo : 0; key < hi;) {
        const int pg = key_page(a, (int)key);
        if ((uint32_t)a.table[b * a.table_s + pg] < (uint32_t)a.pages) return true;
        key = ((int64_t)pg + 1) * a.page;
    }
    return false;
}

// What turns a product into a base-2 exponent.  Positive, or NaN as it is given: a
// hidden key's -inf stays -inf under it and the maximum may be taken before it (a scale
// of 0 still gives every key the same weight).  The sign of a head's scale goes into
// q's: flip_q changes both elements of a dword.
__device__ __forceinline__ float score_scale(const AttendArgs &a, bool f8, int hk)
{
    const float x = __builtin_fabsf(a.scale * (f8 ? a.k_scale[hk] : 1.f) * ATT_LOG2E);
    return x < 1e-37f ? 1e-37f : x;
}
__device__ __forceinline__ int4_t flip_q(const AttendArgs &a, int hk, int4_t q)
{
    const int flip = a.k_scale[hk] < 0.f ? (int)0x80008000u : 0;
    return q ^ int4_t{flip, flip, flip, flip};
}

// ---------------------------------------------------------------------------
// Few query rows for each key head (decode, short chunks): every key is used by
// at most 16 QT rows, so the cache's bytes bound it.  A workgroup takes one
// (sequence, key head, block of 16 QT rows, split of the keys); its waves take
// blocks of 32 keys in turn, each with its own running softmax, and are joined
// in LDS at the end.  Nothing goes through LDS before: 
//   S^T = K Q^T   the A operand of v_mfma_f32_16x16x32 is 8 consecutive elements
//                 of one key: a 16-byte load.
//   O^T = V^T P^T the contraction runs over keys in any order, so P leaves the
//                 first product's accumulators (lane group g: keys 4g .. 4g+3 of
//                 either half of the block) as the second one's B operand.  A
//                 lane loads the same 8 keys' elements 8c .. 8c+7 (c = lane % 16)
//                 and pairs them by v_perm_b32: tile x of the product holds rows
//                 d = 8c + x.
// Pages of a multiple of 16 tokens (P16): each half of a block lies in one page,
// addressed by a buffer resource that ends at the last key of the range: what
// lies behind it reads as zeros.  Other page sizes take a lane's key from its
// own page; the rows' offsets are computed once for each key and handed round.
// Measured: 64 users of up to 8192 keys, 8 key heads of 128 for 32, fp16: 203 us,
// 5.2 TB/s (a plain streaming read of 1 GB reaches 7.1); 4 of up to 131071, e4m3: 167 us, 5.6 TB/s.
// The registers of two waves a SIMD do not hold D = 256 in fp16 or bf16: 27 are spilled (45
// with other page sizes; 7 with those at D = 128 and three waves).  64 users of up to 4096
// keys, D 256: 375 us, 4.3 TB/s.
// ---------------------------------------------------------------------------
__host__ __device__ constexpr int rows_occupancy(int DP, int QT) { return DP <= 128 && QT == 1 ? 3 : 2; }

template <typename S, bool F8, int DP, bool P16, int QT, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(rows_occupancy(DP, QT), rows_occupancy(DP, QT)))) void attend_rows_kernel(const AttendArgs a)
{
    constexpr int EB = F8 ? 1 : 2;                       // bytes of a cache element
    constexpr int KJ = DP / 32;                          // steps of Q K^T
    constexpr int KL = DP * EB / 64;                     // 16-byte loads of a key tile
    constexpr int VW = DP >= 128 ? 8 : DP / 16;          // elements of a V row in one load
    constexpr int VC = DP / (16 * VW);                   // loads of a V row
    constexpr int VD = VW * EB / 4;                      // dwords of one
    constexpr int XT = DP / 16;                          // O^T tiles
    constexpr int LD = DP + 4;                           // row pitch of the join in LDS
    extern __shared__ __attribute__((aligned(16))) float att_lds[];

    // sequence and head fastest, splits slowest: the blocks of one XCD (every 8th)
    // then hold early and late splits alike, and the last ones to start, most of
    // them past their sequence's end, are over at once
    int id = blockIdx.x;
    const int groups = a.B * a.Hkv, bh = id % groups;
    id /= groups;
    const int rb = id % a.rblocks, split = id / a.rblocks, b = bh / a.Hkv, hk = bh - b * a.Hkv;

    const KeyRange kr = key_range(a, b, rb);
    const int nrow = min(16 * QT, kr.n * a.g - rb * a.rows);     // live rows
    if (nrow <= 0) return;
    const int begin = kr.start + split * a.chunk, end = min(kr.hi, begin + a.chunk);
    if (begin >= end && split > 0) return;

    const int lane = threadIdx.x & 63, wave = wave_id(), g = lane >> 4, c = lane & 15;
    const S tag = (S)0.f;

    // Q: row c of each tile, the elements of step j that the K operand has there
    int4_t q[QT][KJ];
    int vhi[QT], vlo[QT];      // the row's keys: [vlo, vhi)
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        const int r = rb * a.rows + 16 * qt + c;
        const int i = r / a.g, hq = hk * a.g + (r - i * a.g);
        const bool live = 16 * qt + c < nrow;
        vhi[qt] = live ? kr.L - kr.n + i + 1 : 0;
        vlo[qt] = a.window > 0 ? vhi[qt] - a.window : 0;
        const char *row = (const char *)a.q + (int64_t)(kr.t0 + (live ? i : 0)) * a.q_ts + (int64_t)(live ? hq : 0) * a.q_hs;
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
            const int d = F8 ? 64 * (j / 2) + 16 * g + 8 * (j & 1) : 32 * j + 8 * g;
            q[qt][j] = *reinterpret_cast<const int4_t *>(row + (d < a.D ? 2 * d : 0));
            if constexpr (F8) q[qt][j] = flip_q(a, hk, q[qt][j]);
            if (!live || d >= a.D) q[qt][j] = int4_t{0, 0, 0, 0};
        }
    }
    // keys that every row of the block sees: [all_lo, all_hi)
    const int all_hi = kr.L - kr.n + rb * a.rows / a.g + 1;
    const int all_lo = a.window > 0 ? kr.hi - a.window : 0;

    uint32_t koff[KL], voff[8][VC];
#pragma unroll
    for (int j = 0; j < KL; ++j) {
        const uint32_t d = 64 * j + 16 * g;
        koff[j] = d < (uint32_t)(a.D * EB) ? (P16 ? c * a.k_ts : 0u) + d : ATT_OOB;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int x = 0; x < VC; ++x) {
            const int d = 16 * VW * x + VW * c;
            voff[e][x] = d < a.D ? (P16 ? (4 * g + (e & 3)) * a.v_ts : 0u) + (uint32_t)(d * EB) : ATT_OOB;
        }

    const float sl = score_scale(a, F8, hk);
    const char *kbase = (const char *)a.k + (int64_t)hk * a.k_hs, *vbase = (const char *)a.v + (int64_t)hk * a.v_hs;
    const int32_t *table = a.table + (int64_t)b * a.table_s;

    // page of (each half of) block blk: P16 two uniform ids, else the id of key lane % 32
    struct Ids {
        int p[2];
    };
    auto ids_of = [&](int blk) {
        Ids r;
        const int key = begin + 32 * blk;
        if constexpr (P16) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int kk = __builtin_amdgcn_readfirstlane(max(0, min(key + 16 * h, end - 1)));
                r.p[h] = table[key_page(a, kk)];
            }
        } else {
            const int kk = max(0, min(key + (lane & 31), end - 1));
            r.p[0] = table[key_page(a, kk)];
            r.p[1] = 0;
        }
        return r;
    };
    // whether a lane's key (P16: the half) is there and its page is one
    auto live_key = [&](int key, int pid) { return key < end && (uint32_t)pid < (uint32_t)a.pages; };

    int4_t kd[2][KL];
    int vd[8][VC][VD];
    auto load_k = [&](int blk, const Ids &ids) {
        const int key = begin + 32 * blk;
        if constexpr (P16) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int kk = __builtin_amdgcn_readfirstlane(key + 16 * t), pid = __builtin_amdgcn_readfirstlane(ids.p[t]);
                const bool ok = live_key(kk, pid);
                const int at = ok ? kk - key_page(a, kk) * a.page : 0;
                const int64_t off = ok ? (int64_t)pid * a.k_ps + (int64_t)at * a.k_ts : 0;
                const uint32_t len = ok ? (uint32_t)(min(16, end - kk) - 1) * a.k_ts + (uint32_t)(a.D * EB) : 0u;
                const __amdgpu_buffer_rsrc_t r = make_rsrc(kbase + off, len);
#pragma unroll
                for (int j = 0; j < KL; ++j)
                    kd[t][j] = __builtin_bit_cast(int4_t, __builtin_amdgcn_raw_buffer_load_b128(r, koff[j], 0, 0));
            }
        } else {
            const int kk = min(key + (lane & 31), end - 1), pid = live_key(kk, ids.p[0]) ? ids.p[0] : 0;
            const int64_t off = (int64_t)pid * a.k_ps + (int64_t)(kk - key_page(a, kk) * a.page) * a.k_ts;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint32_t lo = (uint32_t)__shfl((int)(uint32_t)off, 16 * t + c), hi = (uint32_t)__shfl((int)(off >> 32), 16 * t + c);
                const char *row = kbase + (int64_t)(((uint64_t)hi << 32) | lo);
#pragma unroll
                for (int j = 0; j < KL; ++j)
                    kd[t][j] = *reinterpret_cast<const int4_t *>(row + (koff[j] == ATT_OOB ? 0u : koff[j]));
            }
        }
    };
    auto load_v = [&](int blk, const Ids &ids) {
        const int key = begin + 32 * blk;
        if constexpr (P16) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int kk = __builtin_amdgcn_readfirstlane(key + 16 * t), pid = __builtin_amdgcn_readfirstlane(ids.p[t]);
                const bool ok = live_key(kk, pid);
                const int at = ok ? kk - key_page(a, kk) * a.page : 0;
                const int64_t off = ok ? (int64_t)pid * a.v_ps + (int64_t)at * a.v_ts : 0;
                const uint32_t len = ok ? (uint32_t)(min(16, end - kk) - 1) * a.v_ts + (uint32_t)(a.D * EB) : 0u;
                const __amdgpu_buffer_rsrc_t r = make_rsrc(vbase + off, len);
#pragma unroll
                for (int e = 4 * t; e < 4 * t + 4; ++e)
#pragma unroll
                    for (int x = 0; x < VC; ++x) {
                        if constexpr (VD == 4) {
                            const int4_t w = __builtin_bit_cast(int4_t, __builtin_amdgcn_raw_buffer_load_b128(r, voff[e][x], 0, 0));
#pragma unroll
                            for (int i = 0; i < 4; ++i) vd[e][x][i] = w[i];
                        } else if constexpr (VD == 2) {
                            const int2v_t w = __builtin_bit_cast(int2v_t, __builtin_amdgcn_raw_buffer_load_b64(r, voff[e][x], 0, 0));
                            vd[e][x][0] = w[0];
                            vd[e][x][1] = w[1];
                        } else {
                            vd[e][x][0] = (int)__builtin_amdgcn_raw_buffer_load_b32(r, voff[e][x], 0, 0);
                        }
                    }
            }
        } else {
            const int kk = min(key + (lane & 31), end - 1), pid = live_key(kk, ids.p[0]) ? ids.p[0] : 0;
            const int64_t off = (int64_t)pid * a.v_ps + (int64_t)(kk - key_page(a, kk) * a.page) * a.v_ts;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int src = 16 * (e >> 2) + 4 * g + (e & 3);
                const uint32_t lo = (uint32_t)__shfl((int)(uint32_t)off, src), hi = (uint32_t)__shfl((int)(off >> 32), src);
                const char *row = vbase + (int64_t)(((uint64_t)hi << 32) | lo);
#pragma unroll
                for (int x = 0; x < VC; ++x) {
                    const char *p = row + (voff[e][x] == ATT_OOB ? 0u : voff[e][x]);
                    if constexpr (VD == 4) {
                        const int4_t w = *reinterpret_cast<const int4_t *>(p);
#pragma unroll
                        for (int i = 0; i < 4; ++i) vd[e][x][i] = w[i];
                    } else if constexpr (VD == 2) {
                        const int2v_t w = *reinterpret_cast<const int2v_t *>(p);
                        vd[e][x][0] = w[0];
                        vd[e][x][1] = w[1];
                    } else {
                        vd[e][x][0] = *reinterpret_cast<const int *>(p);
                    }
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
            const int key0 = begin + 32 * blk;
            float4_t s[QT][2];
#pragma unroll
            for (int qt = 0; qt < QT; ++qt)
#pragma unroll
                for (int t = 0; t < 2; ++t) s[qt][t] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int j = 0; j < KJ; ++j) {
                    int4_t kf;
                    if constexpr (F8) {
                        const int w0 = kd[t][j / 2][2 * (j & 1)], w1 = kd[t][j / 2][2 * (j & 1) + 1];
                        kf = int4_t{widen<false>(w0, tag), widen<true>(w0, tag), widen<false>(w1, tag), widen<true>(w1, tag)};
                    } else {
                        kf = kd[t][j];
                    }
#pragma unroll
                    for (int qt = 0; qt < QT; ++qt) s[qt][t] = mfma_16(kf, q[qt][j], s[qt][t], tag);
                }
            // the next block's keys load under this block's softmax and second product
            load_k(blk + NW, nxt);

            bool bad[2];
            if constexpr (P16) {
#pragma unroll
                for (int t = 0; t < 2; ++t) bad[t] = (uint32_t)cur.p[t] >= (uint32_t)a.pages;
            } else {
                // a bad page anywhere in the block: handled key by key below
                bad[0] = bad[1] = __any((uint32_t)cur.p[0] >= (uint32_t)a.pages);
            }
            const bool masked = key0 + 32 > min(all_hi, end) || key0 < all_lo || bad[0] || bad[1];
            if (masked) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int key = key0 + 16 * t + 4 * g + i;
                        bool off = bad[t];
                        if constexpr (!P16) off = (uint32_t)__shfl(cur.p[0], 16 * t + 4 * g + i) >= (uint32_t)a.pages;
#pragma unroll
                        for (int qt = 0; qt < QT; ++qt)
                            if (off || key >= min(vhi[qt], end) || key < vlo[qt]) s[qt][t][i] = -INFINITY;
                        // values that no row sees may hold anything: they meet p = 0 as zeros
                        if (off || key >= end || key < kr.lo) {
#pragma unroll
                            for (int x = 0; x < VC; ++x)
#pragma unroll
                                for (int w = 0; w < VD; ++w) vd[4 * t + i][x][w] = 0;
                        }
                    }
            }
            int4_t p[QT];
#pragma unroll
            for (int qt = 0; qt < QT; ++qt) {
                float x[8], mx = -INFINITY;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] = s[qt][e >> 2][e & 3] * sl;
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
                const float base = ms - ATT_TOP<S>;
                float sum = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] = __builtin_amdgcn_exp2f(x[e] - base);
                    sum += x[e];
                }
                l[qt] += sum;
                p[qt] = int4_t{pack2(x[0], x[1], tag), pack2(x[2], x[3], tag), pack2(x[4], x[5], tag), pack2(x[6], x[7], tag)};
            }
#pragma unroll
            for (int x = 0; x < VC; ++x)
#pragma unroll
                for (int w = 0; w < VW / 2; ++w) {
                    // dword w of the 8 rows (elements 2w, 2w + 1): pair the rows
                    int r[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if constexpr (F8)
                            r[e] = (w & 1) ? widen<true>(vd[e][x][w >> 1], tag) : widen<false>(vd[e][x][w >> 1], tag);
                        else
                            r[e] = vd[e][x][w];
                    }
                    int4_t lo, hi;
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        lo[y] = (int)__builtin_amdgcn_perm((uint32_t)r[2 * y + 1], (uint32_t)r[2 * y], 0x05040100u);
                        hi[y] = (int)__builtin_amdgcn_perm((uint32_t)r[2 * y + 1], (uint32_t)r[2 * y], 0x07060302u);
                    }
#pragma unroll
                    for (int qt = 0; qt < QT; ++qt) {
                        o[qt][VW * x + 2 * w] = mfma_16(lo, p[qt], o[qt][VW * x + 2 * w], tag);
                        o[qt][VW * x + 2 * w + 1] = mfma_16(hi, p[qt], o[qt][VW * x + 2 * w + 1], tag);
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
    const float vs = F8 ? a.v_scale[hk] : 1.f;
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
        bool none = false;
        if (!(tot > 0.f)) {     // (of a split only NaN: whether the others have a sum, the join sees)
            const int hi = kr.L - kr.n + i + 1, lo = a.window > 0 ? hi - a.window : 0;
            none = (a.splits > 1 && tot == 0.f) || !sees_key(a, b, max(begin, lo), min(end, hi));
            tot = NAN;
        }
        const float inv = none ? 0.f : vs / tot;
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = none ? 0.f : sum[e] * inv;
        const float lse2 = none ? -INFINITY : mm - ATT_TOP<S> + __builtin_amdgcn_logf(tot);
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
// Many query rows for each key head (prompts, chunks): bound by the MFMA and the
// clock it leaves, with the softmax's VALU work beside it.  A workgroup of NW waves
// takes 32 NW rows of one (sequence, key head) and one split of the keys; the waves
// share tiles of keys and values in LDS (double-buffered, one barrier a tile), each
// with its own 32 rows: Q^T as B operands, O^T and the statistics in registers.
//   S^T = K Q^T (32x32x16): the A operand is 8 consecutive elements of a key.
//   O^T = V^T P^T: as in the rows kernel the contraction takes the keys in the
//   order in which the first product leaves them (slot (h, e) of step u is key
//   16 u + 8 (e / 4) + 4 h + e % 4), so P goes from accumulators to B operand
//   in registers; the A operand comes from ds_read_b64_tr_b16, which hands 16
//   lanes the columns of a 4 x 16 block of V rows.
// Rows in LDS are DP elements without padding; their 16-byte chunks are XOR-ed
// with a function of the key, so that the 64 banks (256 bytes) are all used: by
// 16 lanes that read one chunk of 16 keys of K, and by 32 lanes that read four
// chunks of 4 keys of V (with XORs that reach 8 chunks only, every read took
// twice its time).
// The maximum is raised only when a tile's exceeds it by more than 2^4: O and l are
// rarely scaled, and nothing else changes.  fp16 probabilities then keep 2^25 below the
// largest in full and are off by 2^-36 of it beyond.
// Measured on two prompts of 4096 tokens, 32 heads of 128, fp16 (cycles of an XCD):
// LDS operands read one by one as the compiler places them 899k, read ahead in
// rings 799k, row places by one key a lane instead of scalar address chains 724k
// (348 us), looked up once for all waves 334 us: 823 TFLOP/s.  In the form before, of
// 335 us (on a card with a higher clock) 67 went with the loads, their stores to LDS and
// the K reads, 20 with the V reads, 26 with the softmax; the MFMAs and the barriers alone
// took 222, twice the time of the instruction's nominal rate (a large fp16 matrix product
// reaches 1159 TFLOP/s).  Slower: the two waves of a SIMD in alternate phases with two
// barriers a tile (356 against 335), one pair's row blocks on one XCD (387), 256
// workgroups with equal stretches of all tiles (453 against 334: row blocks of a head then
// no longer read the same keys at the same time).  No change: raised wave priorities for
// the products.
// ---------------------------------------------------------------------------
typedef float float16v_t __attribute__((ext_vector_type(16)));
typedef short short4v_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float16v_t mfma_32(int4_t a, int4_t b, float16v_t c, _Float16)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
}
__device__ __forceinline__ float16v_t mfma_32(int4_t a, int4_t b, float16v_t c, bf16_t)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8x_t, a), __builtin_bit_cast(bf8x_t, b), c, 0, 0, 0);
}

// keys of a tile: 64, and 32 beyond D = 128, where O^T and Q^T leave no registers for more
__host__ __device__ constexpr int tiles_keys(int D) { return D <= 128 ? 64 : 32; }
constexpr float ATT_LAZY = 4.f;        // a maximum may be exceeded by this much (base 2)

template <typename S, bool F8, int DC, int NW>
__global__ __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(DC <= 128 ? 2 : 1, DC <= 128 ? 2 : 1))) void attend_tiles_kernel(const AttendArgs a)
{
    constexpr int DP = DC == 96 ? 128 : DC;              // pitch of a row in LDS; DC elements of it are computed
    constexpr int KB = tiles_keys(DP), KT = KB / 32;     // keys of a tile, halves of 32 of them
    constexpr int EB = F8 ? 1 : 2;
    constexpr int CH = DP / 8;                           // 16-byte chunks of a row in LDS
    constexpr int LN = KB * CH / (64 * NW);          // chunks of K (and of V) a thread stages
    constexpr int QJ = DC / 16, XT = DC / 32;
    constexpr int TILE = KB * DP * 2;                // bytes
    constexpr float TOP = ATT_TOP<S> > 0.f ? ATT_TOP<S> - ATT_LAZY : 0.f;
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

    const KeyRange kr = key_range(a, b, rb);
    const int nrow = min(32 * NW, kr.n * a.g - rb * a.rows);
    if (nrow <= 0) return;
    const int begin = kr.start + split * a.chunk, end = min(kr.hi, begin + a.chunk);
    if (begin >= end && split > 0) return;

    const int tid = threadIdx.x, lane = tid & 63, wave = wave_id(), c = lane & 31, h = lane >> 5;
    const S tag = (S)0.f;

    // this lane's row
    const int r = rb * a.rows + 32 * wave + c, i = r / a.g, hq = hk * a.g + (r - i * a.g);
    const bool live = 32 * wave + c < nrow;
    const int vhi = live ? kr.L - kr.n + i + 1 : 0, vlo = a.window > 0 ? vhi - a.window : 0;
    int4_t q[QJ];
    {
        const char *row = (const char *)a.q + (int64_t)(kr.t0 + (live ? i : 0)) * a.q_ts + (int64_t)(live ? hq : 0) * a.q_hs;
#pragma unroll
        for (int j = 0; j < QJ; ++j) {
            const int d = 16 * j + 8 * h;
            q[j] = *reinterpret_cast<const int4_t *>(row + (d < a.D ? 2 * d : 0));
            if constexpr (F8) q[j] = flip_q(a, hk, q[j]);
            if (!live || d >= a.D) q[j] = int4_t{0, 0, 0, 0};
        }
    }
    // keys that some row of the wave sees, and keys that all of them see
    const int wr0 = rb * a.rows + 32 * wave, wr1 = min(wr0 + 31, rb * a.rows + nrow - 1);
    const bool wlive = 32 * wave < nrow;
    const int whi = wlive ? kr.L - kr.n + wr1 / a.g + 1 : 0, wall_hi = wlive ? kr.L - kr.n + wr0 / a.g + 1 : 0;
    const int wlo = a.window > 0 ? wall_hi - a.window : 0, wall_lo = a.window > 0 ? whi - a.window : 0;

    const float sl = score_scale(a, F8, hk);
    const char *kbase = (const char *)a.k + (int64_t)hk * a.k_hs, *vbase = (const char *)a.v + (int64_t)hk * a.v_hs;
    const int32_t *table = a.table + (int64_t)b * a.table_s;

    // Where the rows stand: every NW tiles each wave looks up one of the NW tiles after
    // the current ones, lane l the key number l of it, and leaves the key's place in both
    // caches in LDS (2 NW slots), with two masks: keys that some row may see, keys on
    // bad pages.  A key past the end takes the last one's place and a bad page id page
    // 0's: in bounds, and hidden.
    constexpr int SLOTS = 2 * NW;
    int4_t *places = reinterpret_cast<int4_t *>(att_tiles + 4 * TILE);                 // [SLOTS][KB]: K low, high, V low, high
    int4_t *masks = places + SLOTS * KB;                                               // [SLOTS]: seen low, high, bad low, high
    auto key_of = [&](int tile) { return max(0, min(begin + KB * tile + (lane & (KB - 1)), end - 1)); };
    auto ids_of = [&](int tile) { return table[key_page(a, key_of(tile))]; };
    auto look_up = [&](int tile, int pid) {
        const int key = begin + KB * tile + (lane & (KB - 1)), at = key_of(tile) - key_page(a, key_of(tile)) * a.page;
        const bool ok = (uint32_t)pid < (uint32_t)a.pages;
        const uint64_t seen = __ballot(ok && key >= kr.lo && key < end), bad = __ballot(!ok);
        const int pg = ok ? pid : 0, slot = tile % SLOTS;
        const int64_t ko = (int64_t)pg * a.k_ps + (int64_t)at * a.k_ts, vo = (int64_t)pg * a.v_ps + (int64_t)at * a.v_ts;
        if (lane < KB) places[slot * KB + lane] = int4_t{(int)(uint32_t)ko, (int)(ko >> 32), (int)(uint32_t)vo, (int)(vo >> 32)};
        if (lane == 0) masks[slot] = int4_t{(int)(uint32_t)seen, (int)(uint32_t)(seen >> 32), (int)(uint32_t)bad, (int)(uint32_t)(bad >> 32)};
    };
    const int srow = tid / CH, sp = tid % CH;             // this thread stages rows srow + SSTEP n, chunk sp
    constexpr int SSTEP = 64 * NW / CH;
    constexpr int PD = EB * 2;                            // dwords of a piece
    const int in_row = 8 * sp < a.D ? 8 * EB * sp : 0;
    int kst[LN][PD], vst[LN][PD];
    uint64_t vlive = 0, hidden = 0;                       // the masks of the staged tile
    auto uniform64 = [](int lo, int hi) {
        return ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane(hi) << 32) | (uint32_t)__builtin_amdgcn_readfirstlane(lo);
    };
    auto load_tile = [&](int tile) {
        const int slot = tile % SLOTS;
        const int4_t mk = masks[slot];
#pragma unroll
        for (int n = 0; n < LN; ++n) {
            const int4_t at = places[slot * KB + srow + SSTEP * n];
            auto load = [&](const char *src, int (&dst)[PD]) {
                if constexpr (PD == 4) {
                    const int4_t w = *reinterpret_cast<const int4_t *>(src);
#pragma unroll
                    for (int e = 0; e < 4; ++e) dst[e] = w[e];
                } else {
                    const int2v_t w = *reinterpret_cast<const int2v_t *>(src);
                    dst[0] = w[0];
                    dst[1] = w[1];
                }
            };
            load(kbase + (int64_t)(((uint64_t)(uint32_t)at[1] << 32) | (uint32_t)at[0]) + in_row, kst[n]);
            load(vbase + (int64_t)(((uint64_t)(uint32_t)at[3] << 32) | (uint32_t)at[2]) + in_row, vst[n]);
        }
        vlive = uniform64(mk[0], mk[1]);
        hidden = uniform64(mk[2], mk[3]);
    };
    auto store_tile = [&](int buf) {
        auto put = [&](const int (&w)[PD], uint8_t *dst) {
            if constexpr (F8)
                *reinterpret_cast<int4_t *>(dst) = int4_t{widen<false>(w[0], tag), widen<true>(w[0], tag), widen<false>(w[1], tag), widen<true>(w[1], tag)};
            else
                *reinterpret_cast<int4_t *>(dst) = int4_t{w[0], w[1], w[2], w[3]};
        };
        if (~vlive) {     // what a row must not see may hold anything: it meets p = 0 as zeros
#pragma unroll
            for (int n = 0; n < LN; ++n)
#pragma unroll
                for (int e = 0; e < PD; ++e) vst[n][e] = (vlive >> (srow + SSTEP * n)) & 1 ? vst[n][e] : 0;
        }
#pragma unroll
        for (int n = 0; n < LN; ++n) {
            const int row = srow + SSTEP * n;
            put(kst[n], att_tiles + buf * TILE + row * DP * 2 + 16 * (sp ^ swizzle_k(row)));
            put(vst[n], att_tiles + (2 + buf) * TILE + row * DP * 2 + 16 * (sp ^ swizzle_v(row)));
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
        const int buf = tile & 1, key0 = begin + KB * tile;
        load_tile(tile + 1);
        if (tile % NW == 0) {
            look_up(tile + NW + wave, pid);
            pid = ids_of(tile + 2 * NW + wave);
        }
        if (key0 < whi && key0 + KB > wlo) {
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
                s[n / QJ] = mfma_32(kf[n % KA], q[n % QJ], s[n / QJ], tag);
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
            if (key0 + KB > min(wall_hi, end) || key0 < wall_lo || bad) {
                // element e of tile t is key key0 + 4 h + kt, kt a constant
                const int to = min(vhi, end) - key0 - 4 * h, from = vlo - key0 - 4 * h;
                const uint64_t hide = bad >> (4 * h);
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int kt = 32 * t + (e & 3) + 8 * (e >> 2);
                        const bool off = kt >= to || kt < from || ((uint32_t)(hide >> (32 * t)) & (1u << (kt & 31)));
                        s[t][e] = off ? -INFINITY : s[t][e];
                    }
            }
            float mx = s[0][0];
#pragma unroll
            for (int e = 1; e < 16 * KT; ++e) mx = fmaxf(mx, s[e >> 4][e & 15]);
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            mx *= sl;
            if (__any(mx > m + ATT_LAZY)) {              // also the first finite maximum: m is -inf
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
                for (int e = 0; e < 4; ++e) p[e] = pack2(s[u >> 1][8 * (u & 1) + 2 * e], s[u >> 1][8 * (u & 1) + 2 * e + 1], tag);
#pragma unroll
                for (int x = 0; x < XT; ++x) {
                    const int n = u * XT + x;
                    o[x] = mfma_32(vf[n % VA], p, o[x], tag);
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
    bool none = false;
    if (!(l > 0.f)) {     // (of a split only NaN: whether the others have a sum, the join sees)
        none = (a.splits > 1 && l == 0.f) || !sees_key(a, b, max(begin, vlo), min(end, vhi));
        l = NAN;
    }
    const float inv = none ? 0.f : (F8 ? a.v_scale[hk] : 1.f) / l;
    const float lse2 = none ? -INFINITY : m - TOP + __builtin_amdgcn_logf(l);
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

// Joins the splits.  Split s of a row (token, query head) holds the attention
// over its own keys, normalised, and the base-2 log of its sum.  JW waves take
// a row; a wave reads 64 / (DP / 4) splits at once, each lane 4 elements of its
// split, so a row's loads do not wait for each other.
template <typename S, int DP, int JW>
__global__ __launch_bounds__(256) void attend_join_kernel(const AttendArgs a)
{
    constexpr int LN = DP / 4, SW = 64 / LN;        // lanes of a split, splits of a wave
    constexpr int RG = 4 / JW;                      // rows of the workgroup
    __shared__ __attribute__((aligned(16))) float sums[4][DP];
    __shared__ float tots[4];
    const int per = (int)(((int64_t)a.max_q * a.Hq + RG - 1) / RG);
    const int b = blockIdx.x / per, wave = wave_id(), part_wave = wave % JW, lane = threadIdx.x & 63;
    const int r = (blockIdx.x - b * per) * RG + wave / JW, i = r / a.Hq, hq = r - i * a.Hq;
    const int rb = (min(i, a.max_q - 1) * a.g + hq % a.g) / a.rows;
    const KeyRange kr = key_range(a, b, rb);
    const bool live = i < a.max_q && i < kr.n;
    if (JW == 4 && !live) return;                    // the whole workgroup
    const int splits = live ? max(1, (max(0, kr.hi - kr.start) + a.chunk - 1) / a.chunk) : 0;
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
    bool none = false;
    if (!(tot > 0.f)) {
        const int hi = kr.L - kr.n + i + 1, lo = a.window > 0 ? hi - a.window : 0;
        none = !sees_key(a, b, lo, min(kr.L, hi));
        tot = NAN;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = none ? 0.f : sum[e] * (1.f / tot);
    if (lane < LN && d < a.D)
        *reinterpret_cast<int2v_t *>((char *)a.out + (int64_t)(kr.t0 + i) * a.o_ts + (int64_t)hq * a.o_hs + 2 * d) =
            int2v_t{pack2(sum[0], sum[1], (S)0.f), pack2(sum[2], sum[3], (S)0.f)};
    if (a.lse && lane == 0) a.lse[row] = none ? -INFINITY : (mm + __builtin_amdgcn_logf(tot)) * ATT_LN2;
}

// waves of a tiles workgroup: two a SIMD up to D = 128 (256 registers each), one
// beyond (O^T and Q^T alone take 192)
__host__ __device__ constexpr int tiles_waves(int D) { return D <= 128 ? 8 : 4; }
constexpr int ROWS_NW = 4;     // waves of a rows workgroup

int64_t plan_attend(AttendArgs &a, bool e4m3)
{
    // key / page by one multiplication: with l = ceil(log2 page), mul = floor(2^(31+l) / page) + 1
    // is exact for keys below 2^31 (mul page - 2^(31+l) <= page <= 2^l)
    int lg = 0;
    while ((int64_t(1) << lg) < a.page) ++lg;
    a.page_mul = (uint32_t)((uint64_t(1) << (31 + lg)) / (uint64_t)a.page + 1);
    a.page_sh = 31 + lg;

    const int64_t rows = (int64_t)a.max_q * a.g;
    const bool tiles = rows > 32;
    a.rows = tiles ? 32 * tiles_waves(a.D) : rows <= 16 || a.D > 128 ? 16 : 32;
    a.rblocks = (int)((rows + a.rows - 1) / a.rows);
    const int64_t span = 15 + (a.window > 0 ? std::min<int64_t>(a.max_kv, (int64_t)a.window + (a.rows + a.g - 1) / a.g) : a.max_kv);
    const int64_t groups = (int64_t)a.B * a.Hkv * a.rblocks;
    int64_t splits, unit;
    if (tiles) {
        // One workgroup a CU where rows alone do not give them, with at least 320 keys
        // each, two with at least 2048: every split costs 8 bytes of fp32 sums for each
        // output (us: 50 tokens on 48752 keys, one key head of 2: 24 in 152 shares, 62 in 23;
        // 15 x 124 tokens on up to 3078 keys, 4 heads of one: 39 in 8, 97 in one; 600 tokens,
        // 8 heads of 4: 27 in one, 36 in two).
        unit = 128;
        splits = std::max(std::min(256 / groups, span / 320), std::min((512 + groups - 1) / groups, span / 2048));
    } else {
        // A workgroup alone draws about 50 GB/s, so the keys are shared out early: one
        // workgroup a CU with at least 64 KB of keys and values each, two with at least
        // 128 KB (one sequence, 8 key heads of 128, fp16, us: 8000 keys in 64 shares 14.2,
        // in 32 12.9; 1000 keys in 8 shares 8.6, in 4 9.6, in one 12.7).  Shares beyond
        // 2.25 MB are cut into equal parts, so that their number stays a multiple of what
        // the GPU holds at once (4 sequences of up to 131071 keys, e4m3: 167 us in 16
        // shares of 2.1 MB, 177 in 32, 199 in 17; 64 of up to 8192: 203 in two shares of 2 MB,
        // 222 in one).  One launch without a join is enough where the keys are few (300:
        // 7.1 us against 8.6; 513: 9.1 and 8.7) or the groups fill the GPU (32 sequences
        // of up to 2048: 35 and 39 us).
        unit = 32 * ROWS_NW;
        const int64_t bytes = (span - 15) * 2 * a.D * (e4m3 ? 1 : 2), kb = 1024;
        splits = std::max(std::min(256 / groups, (bytes + 64 * kb - 1) / (64 * kb)),
                          std::max<int64_t>(1, std::min((512 + groups - 1) / groups, (bytes + 128 * kb - 1) / (128 * kb))));
        splits *= (std::max<int64_t>(1, bytes / splits) + 2304 * kb - 1) / (2304 * kb);
        if (bytes <= std::max<int64_t>(224, std::min<int64_t>(1024, 4 * groups)) * kb) splits = 1;
    }
    splits = std::max<int64_t>(1, splits);
    a.chunk = (int)(((span + splits - 1) / splits + unit - 1) / unit * unit);
    a.splits = (int)((span + a.chunk - 1) / a.chunk);
    return a.splits > 1 ? (int64_t)a.T * a.Hq * a.splits * (a.D + 1) * 4 : 0;
}

template <typename S, bool F8, int DC>
static hipError_t tiles_go(const AttendArgs &a, hipStream_t st)
{
    constexpr int DP = DC == 96 ? 128 : DC, NW = tiles_waves(DP);
    static bool attr_set = false;
    const size_t lds = (size_t)4 * tiles_keys(DP) * DP * 2 + 2 * NW * (tiles_keys(DP) + 1) * 16;   // tiles, places, masks
    if (!attr_set) {
        hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(&attend_tiles_kernel<S, F8, DC, NW>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
        if (e != hipSuccess) return e;
        attr_set = true;
    }
    hipLaunchKernelGGL((attend_tiles_kernel<S, F8, DC, NW>), dim3((unsigned)((int64_t)a.B * a.rblocks * a.Hkv * a.splits)),
                       dim3(64 * NW), lds, st, a);
    return hipGetLastError();
}

template <typename S, bool F8, int DP, bool P16, int QT>
static hipError_t rows_go(const AttendArgs &a, hipStream_t st)
{
    constexpr int NW = ROWS_NW;
    static bool attr_set = false;
    const int nrow = (int)std::min<int64_t>(16 * QT, (int64_t)a.max_q * a.g);
    const size_t lds = (size_t)NW * nrow * (DP + 6) * 4;
    if (!attr_set) {
        hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(&attend_rows_kernel<S, F8, DP, P16, QT, NW>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
        if (e != hipSuccess) return e;
        attr_set = true;
    }
    hipLaunchKernelGGL((attend_rows_kernel<S, F8, DP, P16, QT, NW>), dim3((unsigned)((int64_t)a.B * a.rblocks * a.Hkv * a.splits)),
                       dim3(64 * NW), lds, st, a);
    return hipGetLastError();
}

template <typename S, bool F8, int DP, bool P16>
static hipError_t rows_pick(const AttendArgs &a, hipStream_t st)
{
    if constexpr (DP <= 128) {
        if (a.rows == 32) return rows_go<S, F8, DP, P16, 2>(a, st);
    }
    return rows_go<S, F8, DP, P16, 1>(a, st);
}

// A wave a row where the splits are few, the workgroup's four where a single
// wave would read them in more than four rounds.
static int join_waves(const AttendArgs &a) { return a.splits <= 4 * (256 / (a.D <= 64 ? 64 : a.D <= 128 ? 128 : 256)) ? 1 : 4; }
static int64_t join_blocks(const AttendArgs &a)     // for each sequence
{
    const int64_t rows = (int64_t)a.max_q * a.Hq;
    return join_waves(a) == 1 ? (rows + 3) / 4 : rows;
}
template <typename S, int DP>
static hipError_t join_go(const AttendArgs &a, hipStream_t st)
{
    const dim3 grid((unsigned)(join_blocks(a) * a.B));
    if (join_waves(a) == 1)
        hipLaunchKernelGGL((attend_join_kernel<S, DP, 1>), grid, dim3(256), 0, st, a);
    else
        hipLaunchKernelGGL((attend_join_kernel<S, DP, 4>), grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

template <typename S, bool F8>
static hipError_t attend_type(const AttendArgs &a, hipStream_t st)
{
    hipError_t e;
    const bool p16 = a.page % 16 == 0;
    if (a.rows > 32)
        e = a.D <= 64 ? tiles_go<S, F8, 64>(a, st) : a.D <= 96 ? tiles_go<S, F8, 96>(a, st)
                      : a.D <= 128 ? tiles_go<S, F8, 128>(a, st) : tiles_go<S, F8, 256>(a, st);
    else if (a.D <= 64)
        e = p16 ? rows_pick<S, F8, 64, true>(a, st) : rows_pick<S, F8, 64, false>(a, st);
    else if (a.D <= 128)
        e = p16 ? rows_pick<S, F8, 128, true>(a, st) : rows_pick<S, F8, 128, false>(a, st);
    else
        e = p16 ? rows_pick<S, F8, 256, true>(a, st) : rows_pick<S, F8, 256, false>(a, st);
    if (e != hipSuccess || a.splits == 1) return e;
    if (a.D <= 64) return join_go<S, 64>(a, st);
    if (a.D <= 128) return join_go<S, 128>(a, st);
    return join_go<S, 256>(a, st);
}

// A launch takes fewer than 2^32 threads.  Both launches of a call are looked at before
// the first: a call is made whole or not at all.
static bool attend_fits(const AttendArgs &a)
{
    const int64_t most = (int64_t(1) << 32) - 1, groups = (int64_t)a.B * a.Hkv;
    const int64_t threads = 64 * (a.rows > 32 ? tiles_waves(a.D) : ROWS_NW);
    if (groups > most || a.rblocks * groups > most / threads / a.splits) return false;
    return a.splits == 1 || join_blocks(a) <= most / 256 / a.B;
}

hipError_t launch_attend(const AttendArgs &a, bool bf16, bool e4m3, hipStream_t st)
{
    if (!attend_fits(a)) return hipErrorNotSupported;
    if (bf16) return e4m3 ? attend_type<bf16_t, true>(a, st) : attend_type<bf16_t, false>(a, st);
    return e4m3 ? attend_type<_Float16, true>(a, st) : attend_type<_Float16, false>(a, st);
}

}  // namespace qmm
