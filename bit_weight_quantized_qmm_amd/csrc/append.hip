// append.hip -- rotary positions on the way into a paged KV cache.
//
// For every token t and head, each rotated pair (a, b) of q and k becomes
//     (a cos - b sin,  b cos + a sin)
// with cos and sin from the fp32 table's row positions[t]; the pairs are
// (i, i + rot/2) or, in the neighbouring form, (2i, 2i+1) for i < rot/2, and
// elements rot .. D-1 pass through.  q goes to `out`, k and v to cache row
// slots[t] (page slot / page_size, row slot % page_size of it), as they are or
// as e4m3 of x / scale[head], saturated at +-448.  Arithmetic in fp32, one
// rounding at the store.
//
// Bound by memory: q, k, v read once and written once.  A thread owns one
// unit, two vectors of V elements (the two halves of V pairs, or 2 V
// neighbours; past rot two vectors that are copied), of one token and of HP
// heads: cos and sin are read once for them.  Neighbouring lanes hold
// neighbouring units, then neighbouring tokens, so a row of 128 is two 128-byte
// stretches.  8192 tokens of 64 + 2 x 8 heads of 128, bf16 (us): with one head a
// thread and the token blocks fastest 84; two heads 81, four 82; with the head
// groups fastest (the table's rows then come from one XCD's L2 once for all
// heads, and a token's heads from one stretch) 72, 65 and 70: 5.2 TB/s.
#include "launch.hpp"
#include "qmm_device.hpp"
#include "elem.hpp"

namespace qmm {

template <int V> struct VecBytes;
template <> struct VecBytes<16> { typedef int4_t t; };
template <> struct VecBytes<8> { typedef int t __attribute__((ext_vector_type(2))); };
template <> struct VecBytes<4> { typedef int t; };
template <> struct VecBytes<2> { typedef short t; };
template <> struct VecBytes<1> { typedef char t; };

template <typename S, int V>
__device__ __forceinline__ void load_vec(const S *p, float (&x)[V])
{
    typedef typename VecBytes<V * sizeof(S)>::t vec;
    S e[V];
    const vec r = *reinterpret_cast<const vec *>(p);
    __builtin_memcpy(e, &r, sizeof r);
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = to_f32(e[i]);
}

template <typename S, int V>
__device__ __forceinline__ void store_vec(S *p, const float (&x)[V])
{
    typedef typename VecBytes<V * sizeof(S)>::t vec;
    S e[V];
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = from_f32<S>(x[i]);
    vec r;
    __builtin_memcpy(&r, e, sizeof r);
    *reinterpret_cast<vec *>(p) = r;
}

template <int V>
__device__ __forceinline__ void load_f32(const float *p, float (&x)[V])
{
    if constexpr (V >= 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4_t r = *reinterpret_cast<const float4_t *>(p + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[i + e] = r[e];
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = p[i];
    }
}

template <typename S, typename C, bool PAIRS, int V, int HP>
__global__ __launch_bounds__(256) void append_kernel(const AppendArgs a)
{
    const int units = a.D / (2 * V);
    // head groups fastest: the blocks that need the same table rows run together
    const int heads = a.Hq + 2 * a.Hkv, hg = (heads + HP - 1) / HP;
    const int tb = (int)(blockIdx.x / (uint32_t)hg), h0 = ((int)blockIdx.x - tb * hg) * HP;
    const int64_t id = (int64_t)tb * 256 + threadIdx.x;
    if (id >= (int64_t)a.T * units) return;
    const int t = (int)((uint32_t)id / (uint32_t)units), u = (int)((uint32_t)id - (uint32_t)t * (uint32_t)units);

    // where the unit's two vectors stand in a row
    const bool turns = u < a.rot / (2 * V);
    const int first = PAIRS || !turns ? 2 * V * u : V * u;
    const int second = PAIRS || !turns ? first + V : first + a.rot / 2;

    const int slot = a.k_cache ? (int)min(max(a.slots[t], (int64_t)-1), (int64_t)0x7fffffff) : -1;
    const bool live = slot >= 0 && slot < a.pages * a.page;
    const int pg = live ? slot / a.page : 0, at = live ? slot - pg * a.page : 0;

    float cs[V], sn[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        cs[i] = 1.f;
        sn[i] = 0.f;
    }
    if (turns) {
        const int pos = min(max(a.positions[t], 0), a.table_rows - 1);
        const float *line = a.rope + (size_t)pos * a.rot + V * u;
        load_f32<V>(line, cs);
        load_f32<V>(line + a.rot / 2, sn);
    }

    float x[HP][2][V];
#pragma unroll
    for (int i = 0; i < HP; ++i) {
        const int h = h0 + i;
        if (h >= heads) break;
        const S *src;
        if (h < a.Hq)
            src = (const S *)a.q + (size_t)t * a.q_ts + (size_t)h * a.q_hs;
        else if (h < a.Hq + a.Hkv)
            src = (const S *)a.k + (size_t)t * a.k_ts + (size_t)(h - a.Hq) * a.k_hs;
        else
            src = (const S *)a.v + (size_t)t * a.v_ts + (size_t)(h - a.Hq - a.Hkv) * a.v_hs;
        load_vec<S, V>(src + first, x[i][0]);
        load_vec<S, V>(src + second, x[i][1]);
    }
#pragma unroll
    for (int i = 0; i < HP; ++i) {
        const int h = h0 + i;
        if (h >= heads) break;
        if (h < a.Hq + a.Hkv) {
            float y[2 * V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                // neighbouring form: pair e is elements 2e, 2e+1 of the 2 V in a row
                const float p = PAIRS ? (2 * e < V ? x[i][0][(2 * e) % V] : x[i][1][(2 * e) % V]) : x[i][0][e];
                const float q = PAIRS ? (2 * e + 1 < V ? x[i][0][(2 * e + 1) % V] : x[i][1][(2 * e + 1) % V]) : x[i][1][e];
                y[PAIRS ? 2 * e : e] = p * cs[e] - q * sn[e];
                y[PAIRS ? 2 * e + 1 : V + e] = q * cs[e] + p * sn[e];
            }
            if (turns) {
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    x[i][0][e] = y[e];
                    x[i][1][e] = y[V + e];
                }
            }
        }
        if (h < a.Hq) {
            S *dst = (S *)a.out + (size_t)t * a.o_ts + (size_t)h * a.o_hs;
            store_vec<S, V>(dst + first, x[i][0]);
            store_vec<S, V>(dst + second, x[i][1]);
        } else if (live) {
            const bool is_k = h < a.Hq + a.Hkv;
            const int hk = is_k ? h - a.Hq : h - a.Hq - a.Hkv;
            C *dst = is_k ? (C *)a.k_cache + (size_t)pg * a.kc_ps + (size_t)hk * a.kc_hs + (size_t)at * a.kc_ts
                          : (C *)a.v_cache + (size_t)pg * a.vc_ps + (size_t)hk * a.vc_hs + (size_t)at * a.vc_ts;
            if constexpr (sizeof(C) == 1) {
                const float sc = (is_k ? a.k_scale : a.v_scale)[hk];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    x[i][0][e] = x[i][0][e] / sc;
                    x[i][1][e] = x[i][1][e] / sc;
                }
            }
            store_vec<C, V>(dst + first, x[i][0]);
            store_vec<C, V>(dst + second, x[i][1]);
        }
    }
}

template <typename S, typename C, bool PAIRS, int V>
static hipError_t append_go(const AppendArgs &a, hipStream_t st)
{
    constexpr int HP = 2;
    const int64_t blocks = ((int64_t)a.T * (a.D / (2 * V)) + 255) / 256 * ((a.Hq + 2 * a.Hkv + HP - 1) / HP);
    if (blocks * 256 >= (int64_t(1) << 32)) return hipErrorNotSupported;   // threads of a launch
    hipLaunchKernelGGL((append_kernel<S, C, PAIRS, V, HP>), dim3((unsigned)blocks), dim3(256), 0, st, a);
    return hipGetLastError();
}

template <typename S, typename C>
static hipError_t append_pick(const AppendArgs &a, int vec, hipStream_t st)
{
    if (a.pairs) {
        if (vec == 8) return append_go<S, C, true, 8>(a, st);
        if (vec == 4) return append_go<S, C, true, 4>(a, st);
        return append_go<S, C, true, 1>(a, st);
    }
    if (vec == 8) return append_go<S, C, false, 8>(a, st);
    if (vec == 4) return append_go<S, C, false, 4>(a, st);
    return append_go<S, C, false, 1>(a, st);
}

// vec: 8, 4 or 1 elements a vector (the caller has checked that every row and
// both vectors of a unit stand at multiples of it)
hipError_t launch_append(const AppendArgs &a, bool bf16, bool e4m3, int vec, hipStream_t st)
{
    if (bf16) return e4m3 ? append_pick<bf16_t, fp8_t>(a, vec, st) : append_pick<bf16_t, bf16_t>(a, vec, st);
    return e4m3 ? append_pick<_Float16, fp8_t>(a, vec, st) : append_pick<_Float16, _Float16>(a, vec, st);
}

}  // namespace qmm
