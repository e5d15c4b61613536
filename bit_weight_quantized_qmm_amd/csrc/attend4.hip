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
// (up to a multiple of 2^lg_unit), then the keys from the block's first window on.
#include <algorithm>
#include <math.h>

#include "attend.hpp"

namespace qmm {

typedef _Float16 f16_t;

// fp16 probabilities are scaled by 2^15: in full down to 2^-29 of a row's largest.
constexpr float A4_TOP = 15.f;
constexpr float A4_LAZY = 4.f;         // a maximum may be exceeded by this much (base 2): p ends at 2^15
constexpr float A4_LIFT = 24.f;        // of weights p s: brings the least s of fp16 to 1

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
    const int first = a.by_g(rb * a.rows), last = a.by_g(max(0, min((rb + 1) * a.rows, n * a.g) - 1));
    r.hi = max(0, min(r.L, r.L - n + last + 1));
    r.lo = a.window > 0 ? max(0, r.L - n + first - a.window + 1) : 0;
    r.sk = min(a.sinks, r.hi);
    r.start = r.lo & ~15;
    r.S = (r.sk + (1 << a.lg_unit) - 1) >> a.lg_unit << a.lg_unit;
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

// whether a scale (and its zero-point) has NaN for a scale
__device__ __forceinline__ bool is_nan(uint32_t sz) { return (sz & 0x7fffu) > 0x7c00u; }

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
// The largest of the sizes of a dword's two elements and of `so_far`'s, as they stand (f16 and bf16 order
// like whole numbers); a half of that as a number.
typedef uint16_t ushort2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t larger2(uint32_t so_far, int4_t q)
{
    ushort2_t m = __builtin_bit_cast(ushort2_t, so_far);
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(ushort2_t, (uint32_t)q[i] & 0x7fff7fffu));
    return __builtin_bit_cast(uint32_t, m);
}
__device__ __forceinline__ float size_of(uint32_t bits, f16_t) { return (float)as_half((uint16_t)bits); }
__device__ __forceinline__ float size_of(uint32_t bits, bf16_t) { return __builtin_bit_cast(float, bits << 16); }
// N steps of a row in codes' order as f16 times 2^up; PART: the elements whose codes stand higher by 16 less
template <bool PART, int N>
__device__ __forceinline__ void scale_row(int4_t (&q)[N], int up, f16_t)
{
    int low = up, high = PART ? up - 4 : up;
    do {                                    // 2^15 at a time: once but for rows below 1
        const f16_t fl = (f16_t)ldexpf(1.f, min(low, 15)), fh = (f16_t)ldexpf(1.f, min(high, 15));
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) q[j][i] = (int)as_u32(as_half2((uint32_t)q[j][i]) * (i & 1 ? half2_t{fh, fh} : half2_t{fl, fl}));
        low = max(low - 15, 0);
        high = max(high - 15, 0);
    } while (__any(low > 0));
}
template <bool PART, int N>
__device__ __forceinline__ void scale_row(int4_t (&q)[N], int up, bf16_t)
{
#pragma unroll
    for (int j = 0; j < N; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int by = PART && (i & 1) ? up - 4 : up;
            const float x = __builtin_bit_cast(float, (uint32_t)q[j][i] << 16), y = __builtin_bit_cast(float, (uint32_t)q[j][i] & 0xffff0000u);
            q[j][i] = pack2(ldexpf(x, by), ldexpf(y, by), f16_t());
        }
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

// The codes of a dword, in codes' order, as f16 without an exponent: c 2^-22, c 2^-18, c 2^-22, c 2^-18.
// The matrix instruction aligns products as if such leading zeros were digits, so its sums lose bits with them.  Worst
// and root mean square of 32 products, as parts of the sum of their sizes, for codes of any size and codes of 1:
//     c 2^-24           2^-18.5  2^-21.3      2^-15.7  2^-18.6
//     c 2^-22, 2^-18    2^-21.6  2^-24.8      2^-18.4  2^-21.8
//     c 2^-20           2^-22.6  2^-26.0      2^-21.2  2^-24.6
//     c                 2^-23.4  2^-26.0      2^-24.8  2^-29.7
// 32 roundings of fp32 in a row are 2^-19 at most.  The first takes one operation less for 8 codes, the third one more
// (64 users of up to 8192 keys, G 64: 71.5 us, the third's 74; 4 of up to 131071, G 128: 97.2 and 98.7).
__device__ __forceinline__ int4_t places4(uint32_t w)
{
    const uint32_t low = w << 2, high = w >> 6;
    return int4_t{(int)(low & 0x003c003cu), (int)(low & 0x03c003c0u), (int)(high & 0x003c003cu), (int)(high & 0x03c003c0u)};
}

// ---------------------------------------------------------------------------
// Few query rows for each key head (decode, short chunks): as attend_rows_kernel, a
// workgroup takes one (sequence, key head, block of 16 QT rows, split of the
// places), its waves take blocks of 32 places in turn, each with its own running
// softmax, and are joined in LDS.
//   S^T = K Q^T   lane (g, c) holds a slice of key c's codes; q stands in the same order.
//   O^T = V^T P^T lane (g, c) holds elements of 8 keys (4g .. 4g + 3 of either half); the
//                 dwords of two keys are put together before the codes are taken out, so
//                 that a pair of f16 is one element of two keys.
// What bounds it is the instructions between a byte of codes and its product, so with
// groups of 64 or 128 (GM) nothing is computed for each code but its mask:
//   K   c at bits 2 .. 5 of a half is the f16 c 2^-22, at bits 6 .. 9 c 2^-18, which the
//       matrix instruction takes as they are; the rows of q, brought to 2^14 .. 2^15, have
//       their elements there divided by 16.  A step of the contraction lies in one group:
//           x = sum over the groups of s (sum_d q_d c_d - z sum_d q_d),
//       on the accumulators, four keys of a lane.
//   V   a tile of O^T lies in one group, whose s goes into the probabilities: p s 2^lift,
//       rounded to f16 as p would be; sum_j p_j s_j z_j is a product of its own, taken off at
//       the end.  Each row has a lift for each group, such that its largest p s there stands at
//       2^11 to 2^15: other groups' scales, and those of keys that get no weight, take none of
//       its bits.  The first group's is in the exponent of p already.  (In groups of 64 the lanes
//       c and c ^ 1 read a dword of two keys each and change halves.)
// Other groups (GM = 32): every code becomes (c - z) s in f16.
// Codes and scales go from memory into LDS without a register, two blocks ahead, each wave into a
// ring of its own; they are read once, so they leave no trace in the L2 (with the default policy the
// loads alone took 95 us of the 4 sequences below, 84 without).
// Pages of a multiple of 16 tokens (HALVES): a half of a block lies in one page; lane l looks
// up the l-th half of the next 32 blocks, and its place goes to scalar registers
// when its turn comes.  Other page sizes: a lane's key by its own page, two blocks a lookup; where
// a page holds a cache line or less of a head (SHARED), a sequence's heads run on one L2, whose lines they share.
// A value of NaN counts as 0 where rows of the block see different keys, and makes its group NaN for the rows that
// see it at the end; where all see it the products do that.
// Measured (us): 4 sequences of up to 131071 keys, 8 key heads of 128 for 64, G 128: 95 to 98 (5.2
// TB/s; the loads alone 85; a plain streaming read reaches 7.1); 64 of up to 8192, 32 heads: G 128 64 (4.4; the loads alone
// 57), G 64 70 to 76 (57; cards differ), G 32 76 (63); one of 513 keys 9.5 (7.4).
// ---------------------------------------------------------------------------
enum { HALVES, ANY, SHARED };         // PAGES
__host__ __device__ constexpr int rows4_occupancy(int DP, int GM, int PAGES, int QT)
{
    return DP > 128 || QT > 1 ? 2 : DP == 128 && (GM == 64 || (GM == 128 && PAGES != HALVES)) ? 3 : 4;
}
__host__ __device__ constexpr int rows4_waves(int DP) { return DP > 128 ? 2 : 4; }      // 64 KB of ring at most
__host__ __device__ constexpr int rows4_groups(int DP, int GM) { return GM > 32 ? DP / GM : DP / 32; }
// bytes of a half's scales in LDS, whole loads of 64 lanes; of a block of 32 places: codes and scales of K and V
__host__ __device__ constexpr int rows4_scales(int DP, int GM) { return rows4_groups(DP, GM) <= 4 ? 256 : 64 * rows4_groups(DP, GM); }
__host__ __device__ constexpr int rows4_block(int DP, int GM) { return 2 * (32 * DP / 2 + 2 * rows4_scales(DP, GM)); }
constexpr int ROWS4_IDS = 8;          // blocks whose page ids a wave keeps in LDS where pages are no multiple of 16 tokens
__host__ __device__ constexpr int rows4_ring(int DP, int GM, int PAGES) { return 2 * rows4_block(DP, GM) + (PAGES == HALVES ? 0 : ROWS4_IDS * 32 * 4); }

// Loads of the lanes' 16 (4) bytes at p + off into LDS, from `to` on, lane by lane.  The compiler does
// not know that they are in flight: wait_loads() before what they bring is read, and what stood there
// must have been read.
template <int BYTES>
__device__ __forceinline__ void fetch(uint32_t to, __amdgpu_buffer_rsrc_t r, uint32_t off)
{
    if constexpr (BYTES == 16)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds" ::"s"(to), "v"(off), "s"(r) : "memory", "m0");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen nt lds" ::"s"(to), "v"(off), "s"(r) : "memory", "m0");
}
template <int BYTES, bool KEEP>
__device__ __forceinline__ void fetch(uint32_t to, const uint8_t *p)
{
    if constexpr (BYTES == 16 && KEEP)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(p) : "memory", "m0");
    else if constexpr (BYTES == 16)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off nt" ::"s"(to), "v"(p) : "memory", "m0");
    else if constexpr (KEEP)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(to), "v"(p) : "memory", "m0");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off nt" ::"s"(to), "v"(p) : "memory", "m0");
}
template <int N> __device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }
__device__ __forceinline__ void wait_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

template <typename S, int DP, int GM, int PAGES, int QT>
__global__ __launch_bounds__(64 * rows4_waves(DP)) __attribute__((amdgpu_waves_per_eu(rows4_occupancy(DP, GM, PAGES, QT), rows4_occupancy(DP, GM, PAGES, QT)))) void attend4_rows_kernel(const Attend4Args a)
{
    constexpr int NW = rows4_waves(DP);
    constexpr bool P16 = PAGES == HALVES, NEAR = PAGES == SHARED;
    constexpr bool DEFER = GM > 32;
    constexpr int KJ = DP / 32;                                   // steps of Q K^T
    constexpr int KW = DEFER ? GM / 32 : DP == 64 ? 2 : 4;        // dwords of a slice
    constexpr int KL = KJ / KW;                                   // slices of a lane: of one group each
    constexpr int VW = GM == 128 ? 8 : GM == 64 ? 4 : DP >= 128 ? 8 : 4;   // elements of a V row that a lane has of a chunk
    constexpr int VC = DP / (16 * VW);                            // chunks of a V row
    constexpr int VK = GM == 64 ? 2 : 4;                          // dwords of a chunk in a half: of a key, or of two
    constexpr int XT = DP / 16;                                   // O^T tiles
    constexpr int NS = DEFER ? DP / GM : 1;                       // groups of a token
    constexpr int NX = rows4_groups(DP, GM);                      // and room for them
    constexpr int CH = DP / 32;                                   // 16-byte pieces of a token's row
    constexpr int HALF = 16 * 16 * CH, SHALF = rows4_scales(DP, GM);      // bytes of a half's codes, scales
    constexpr int CF = CH > 4 ? CH / 4 : 1, SF = NX > 4 ? NX / 4 : 1;   // loads of a half's codes, scales
    constexpr int FETCHES = 2 * (CF + SF);                        // loads of a block's keys, or values
    constexpr int BLOCK = rows4_block(DP, GM);
    constexpr int LD = DP + 4;                                    // row pitch of the join in LDS
    constexpr float TOP = A4_TOP - A4_LAZY;
    extern __shared__ __attribute__((aligned(16))) float att_lds[];

    // head and sequence fastest, splits slowest; SHARED: eight sequences take turns (workgroups go round the
    // eight L2s), so that a sequence's heads share one
    const int id = blockIdx.x, eight = NEAR ? a.by_Hkv(id >> 3) : 0;
    const bool turns = NEAR && (eight + 1) * 8 * a.Hkv <= (int)gridDim.x;
    const int rest = turns ? 8 * eight + (id & 7) : a.by_Hkv(id), hk = turns ? (id >> 3) - eight * a.Hkv : id - rest * a.Hkv;
    const int above = a.by_groups(rest * a.Hkv), b = rest - above * a.B;
    const int split = a.by_rblocks(above), rb = above - split * a.rblocks;

    // Without a window a place is its key, whatever the lengths say: the first pages are looked up
    // while those are on their way.
    const int32_t *table = a.table + (int64_t)b * a.table_s;
    const int lane = threadIdx.x & 63, wave = wave_id(), g = lane >> 4, c = lane & 15;
    const int begin = split * a.chunk;
    int first_id = 0;
    if (P16 && a.window == 0) first_id = table[min(key_page(a, begin + 32 * (wave + NW * (lane >> 1)) + 16 * (lane & 1)), a.width - 1)];

    const Range4 kr = range4(a, b, rb);
    const int nrow = min(16 * QT, kr.n * a.g - rb * a.rows);     // live rows
    if (nrow <= 0) return;
    const int end = min(kr.len, begin + a.chunk);
    if (begin >= end && split > 0) return;
    const S tag = (S)0.f;

    // ---- where a lane's pieces stand ----
    // In LDS a half's K is [piece][key], so that each lane reads what 16 (8) bytes it needs; its V
    // stands such that the dwords that 64 lanes read at once lie in 64 banks: pieces of 16 bytes in
    // the order [group][e][g][c % 2][c / 8] (GM = 64), else [pieces / 4][i][g][piece % 4] (the key is 4g + i, or 4g + 2e +
    // c % 2).
    uint8_t *ring = reinterpret_cast<uint8_t *>(att_lds) + wave * rows4_ring(DP, GM, PAGES);
    const uint32_t ring_at = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)ring);
    int kkey[CF], vkey[CF];                 // of the piece that this lane loads: its key, where in the row
    uint32_t kpart[CF], vpart[CF];
#pragma unroll
    for (int f = 0; f < CF; ++f) {
        const int sl = 64 * f + lane;
        int piece = sl >> 4;
        kkey[f] = sl & 15;
        kpart[f] = 32 * piece < a.D ? 16 * piece : 0;
        if constexpr (GM == 64) {
            vkey[f] = 4 * ((sl >> 2) & 3) + 2 * ((sl >> 4) & 1) + ((sl >> 1) & 1);
            piece = 2 * (sl >> 5) + (sl & 1);
        } else if constexpr (CH == 2) {
            vkey[f] = 4 * ((sl >> 1) & 3) + ((sl >> 3) & 3);
            piece = sl & 1;
        } else {
            vkey[f] = 4 * ((sl >> 2) & 3) + ((sl >> 4) & 3);
            piece = 4 * (sl >> 6) + (sl & 3);
        }
        vpart[f] = 32 * piece < a.D ? 16 * piece : 0;
    }
    const int n_s = DEFER ? NS : (int)(a.s_ts >> 2);                // groups of a token
    const uint32_t *kread = reinterpret_cast<const uint32_t *>(ring) + (KW == 4 ? 64 * g + 4 * c : 64 * (g >> 1) + 4 * c + 2 * (g & 1));
    const uint8_t *vread = ring + 2 * HALF + (GM == 64 ? 16 * (4 * g + 2 * (c & 1) + (c >> 3)) + 4 * ((c >> 1) & 3)
                                                       : CH == 2 ? 16 * (2 * g + (c >> 3)) + (2 * c & 15) : 16 * (4 * g + (c >> 2)) + 4 * (c & 3));
    const uint32_t *kscale = reinterpret_cast<const uint32_t *>(ring + 4 * HALF) + (DEFER ? 4 * NS * g : c * n_s);
    const uint32_t *vscale = reinterpret_cast<const uint32_t *>(ring + 4 * HALF + 2 * SHALF) + 4 * n_s * g;
    int kgroup[KL], vgroup[VC];             // generic: the groups of this lane's slices and chunks
#pragma unroll
    for (int j = 0; j < KL; ++j) kgroup[j] = min(32 * KW * j + 8 * KW * g, a.D - 1) >> a.lg_G;
#pragma unroll
    for (int x = 0; x < VC; ++x) vgroup[x] = min(16 * VW * x + VW * c, a.D - 1) >> a.lg_G;

    const uint8_t *kbase = a.k + (int64_t)hk * a.k_hs, *vbase = a.v + (int64_t)hk * a.v_hs;
    const uint8_t *ksbase = (const uint8_t *)a.ks + (int64_t)hk * a.ks_hs, *vsbase = (const uint8_t *)a.vs + (int64_t)hk * a.vs_hs;
    auto is_page = [&](int pid) { return (uint32_t)pid < (uint32_t)a.pages; };

    // ---- the lookups ----
    // P16: lane l, half l % 2 of this wave's block number 32 n + l / 2; else lane l, place l % 32 of block
    // 2 n + l / 32, the page ids in LDS for ROWS4_IDS blocks.  A place past the end or on a bad page is token
    // 0 of page 0: in bounds, and hidden.
    auto place_of = [&](int n) {
        return P16 ? begin + 32 * (wave + NW * (32 * n + (lane >> 1))) + 16 * (lane & 1) : begin + 32 * (wave + NW * (2 * n + (lane >> 5))) + (lane & 31);
    };
    auto key_of = [&](int v) { return key_at(kr, max(0, min(v, end - 1))); };
    int64_t ko = 0, vo = 0, kso = 0, vso = 0;
    uint64_t dead = 0;                          // lanes whose place is no key
    auto look_up = [&](int n, int pid) {
        const int v = place_of(n), key = key_of(v);
        const bool ok = v < end && is_page(pid);
        const int64_t pg = ok ? pid : 0, at = ok ? key - key_page(a, key) * a.page : 0;
        ko = pg * a.k_ps + at * a.k_ts;
        vo = pg * a.v_ps + at * a.v_ts;
        kso = pg * a.ks_ps + at * a.s_ts;
        vso = pg * a.vs_ps + at * a.s_ts;
        dead = __ballot(!ok);
    };
    int32_t *ids = reinterpret_cast<int32_t *>(ring + 2 * BLOCK);
    auto hold_ids = [&](int n) {                // of blocks n .. n + ROWS4_IDS - 1, n even
        int32_t x[ROWS4_IDS / 2];
#pragma unroll
        for (int i = 0; i < ROWS4_IDS / 2; ++i) x[i] = table[key_page(a, key_of(place_of(n / 2 + i)))];
#pragma unroll
        for (int i = 0; i < ROWS4_IDS / 2; ++i) ids[64 * i + lane] = x[i];
    };
    auto held = [&](int64_t x, int l) {         // lane l's, uniform
        const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)x, l), hi = (uint32_t)__builtin_amdgcn_readlane((int)(x >> 32), l);
        return (int64_t)(((uint64_t)hi << 32) | lo);
    };
    auto sent = [&](int64_t x, int l) {         // lane l's, each lane's own l
        const uint32_t lo = (uint32_t)__shfl((int)(uint32_t)x, l), hi = (uint32_t)__shfl((int)(x >> 32), l);
        return (int64_t)(((uint64_t)hi << 32) | lo);
    };
    // a block's keys or values on their way into its place in the ring (lanes past a half's scales load its last again)
    uint32_t spart[SF];
    int stok[SF];
#pragma unroll
    for (int f = 0; f < SF; ++f) {
        spart[f] = min(64 * f + lane, 16 * n_s - 1);
        stok[f] = (int)spart[f] / n_s;
        spart[f] = P16 ? 4 * spart[f] : 4 * (spart[f] - stok[f] * n_s);
    }
    auto fetch_side = [&](int n, const uint8_t *base, const uint8_t *sbase, int64_t off, int64_t soff, uint32_t ts, const int (&key)[CF], const uint32_t (&part)[CF],
                          uint32_t to, uint32_t sto) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if constexpr (P16) {
                const __amdgpu_buffer_rsrc_t r = make_rsrc(base + held(off, 2 * (n & 31) + t), 0x7fffffffu), rs = make_rsrc(sbase + held(soff, 2 * (n & 31) + t), 0x7fffffffu);
#pragma unroll
                for (int f = 0; f < CF; ++f)
                    if (CH >= 4 || lane < 16 * CH) fetch<16>(to + t * HALF + 1024 * f, r, key[f] * ts + part[f]);
#pragma unroll
                for (int f = 0; f < SF; ++f) fetch<4>(sto + t * SHALF + 256 * f, rs, spart[f]);
            } else {
#pragma unroll
                for (int f = 0; f < CF; ++f) {
                    const uint8_t *p = base + sent(off, 32 * (n & 1) + 16 * t + key[f]) + part[f];
                    if (CH >= 4 || lane < 16 * CH) fetch<16, NEAR>(to + t * HALF + 1024 * f, p);
                }
#pragma unroll
                for (int f = 0; f < SF; ++f) fetch<4, NEAR>(sto + t * SHALF + 256 * f, sbase + sent(soff, 32 * (n & 1) + 16 * t + stok[f]) + spart[f]);
            }
        }
    };
    auto fetch_k = [&](int n) { fetch_side(n, kbase, ksbase, ko, kso, a.k_ts, kkey, kpart, ring_at + (n & 1) * BLOCK, ring_at + (n & 1) * BLOCK + 4 * HALF); };
    auto fetch_v = [&](int n) {
        fetch_side(n, vbase, vsbase, vo, vso, a.v_ts, vkey, vpart, ring_at + (n & 1) * BLOCK + 2 * HALF, ring_at + (n & 1) * BLOCK + 4 * HALF + 2 * SHALF);
    };

    const int all_blocks = (max(0, end - begin) + 31) >> 5;
    const int blocks = all_blocks > wave ? (all_blocks - wave + NW - 1) / NW : 0;      // of this wave
    uint64_t gone[3] = {0, 0, 0};      // places that are no keys, of blocks n, n + 1 and n + 2
    int nid = 0;                       // P16: the next lookup's page ids
    if (blocks > 0) {
        if constexpr (P16) {
            const int first = a.window == 0 ? first_id : table[key_page(a, key_of(place_of(0)))];
            nid = table[key_page(a, key_of(place_of(1)))];
            look_up(0, first);
            gone[0] = dead & 3, gone[1] = dead >> 2 & 3;
            fetch_k(0);
            fetch_v(0);
            fetch_k(1);
            fetch_v(1);
        } else {
            hold_ids(0);
            look_up(0, ids[lane]);
            for (int n = 0; n < 2; ++n) {
                gone[n] = dead >> (32 * n) & 0xffffffffu;
                fetch_k(n);
                fetch_v(n);
            }
        }
    }

    // ---- the rows of q ----
    int4_t q[QT][KJ];
    int vhi[QT], vlo[QT];      // the row's keys: [vlo, vhi), and those below the sinks
    float sl[QT], qsum[QT][NS];
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        const int r = rb * a.rows + 16 * qt + c;
        const int i = a.by_g(r), hq = hk * a.g + (r - i * a.g);
        const bool live = 16 * qt + c < nrow;
        vhi[qt] = live ? kr.L - kr.n + i + 1 : 0;
        vlo[qt] = a.window > 0 ? vhi[qt] - a.window : 0;
        const char *row = (const char *)a.q + (int64_t)(kr.t0 + (live ? i : 0)) * a.q_ts + (int64_t)(live ? hq : 0) * a.q_hs;
        uint32_t bits = 0;
#pragma unroll
        for (int j = 0; j < KJ; ++j) {
            const int d = 32 * KW * (j / KW) + 8 * KW * g + 8 * (j % KW);
            q[qt][j] = *reinterpret_cast<const int4_t *>(row + (d < a.D ? 2 * d : 0));
            if (!live || d >= a.D) q[qt][j] = int4_t{0, 0, 0, 0};
            bits = larger2(bits, q[qt][j]);
        }
        sl[qt] = a.scale * ATT_LOG2E;
#pragma unroll
        for (int j = 0; j < KJ; ++j) q[qt][j] = code_order(q[qt][j]);
        if constexpr (DEFER || !__is_same(S, f16_t)) {
            float top = size_of(max(bits & 0xffffu, bits >> 16), tag);
            top = fmaxf(top, __shfl_xor(top, 16));
            top = fmaxf(top, __shfl_xor(top, 32));
            const int up = rise_of(top);
            scale_row<DEFER, KJ>(q[qt], up, tag);
            sl[qt] = fminf(ldexpf(sl[qt], (DEFER ? 22 : 0) - up), 3e38f);
        }
        sl[qt] = above_zero(sl[qt]);
        if constexpr (DEFER) {
#pragma unroll
            for (int ns = 0; ns < NS; ++ns) {
                // of a key whose codes are all 1; as 1 and 16, which keep all bits (z times it is taken off)
                float4_t sum = float4_t{0.f, 0.f, 0.f, 0.f};
                const int4_t ones = int4_t{0x3c003c00, 0x4c004c00, 0x3c003c00, 0x4c004c00};
#pragma unroll
                for (int w = 0; w < KW; ++w) sum = mfma_16(ones, q[qt][KW * ns + w], sum, f16_t());
                qsum[qt][ns] = sum[0] * 0x1p-22f;
            }
        }
    }
    // rows of different tokens see different keys: a value of NaN is for those that see it
    const bool alike = a.by_g(rb * a.rows) == a.by_g(rb * a.rows + nrow - 1);
    uint32_t spoilt[QT];       // chunk x, place i of 16: bit 16 x + i
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) spoilt[qt] = 0;
    // keys that every row of the block sees: [all_lo, all_hi) (and those below the sinks)
    const int all_hi = min(kr.hi, kr.L - kr.n + a.by_g(rb * a.rows) + 1);
    const int all_lo = a.window > 0 ? kr.hi - a.window : 0;

    // m: the running maximum.  DEFER: rounded down to a whole number, as the lifts are, so that what stands is
    // multiplied by powers of two alone; l and group 0 are in units of 2^(lift[0] - m), group ns' in 2^(lift[ns] - m),
    // `more` times as large (two groups at most)
    float m[QT], l[QT], lift[QT][NS], more[QT];
    float4_t o[QT][XT], oz[QT][NS];      // oz: sum of p s z, alike in all four
#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        m[qt] = -INFINITY;
        l[qt] = 0.f;
        more[qt] = 1.f;
#pragma unroll
        for (int x = 0; x < XT; ++x) o[qt][x] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < NS; ++x) {
            oz[qt][x] = float4_t{0.f, 0.f, 0.f, 0.f};
            lift[qt][x] = A4_LIFT;
        }
    }
    auto scale_group = [&](int qt, int ns, float f) {
#pragma unroll
        for (int x = 0; x < XT / NS; ++x) o[qt][XT / NS * ns + x] *= f;
        oz[qt][ns] *= f;
    };

    for (int n = 0; n < blocks; ++n) {
        const int v0 = begin + 32 * (wave + NW * n);
        const int in_ring = (n & 1) * BLOCK;
        // loads of V n, K n + 1 and V n + 1 stay on their way
        wait_loads<3 * FETCHES>();
        uint32_t kd[2][KL][KW], ksd[2][DEFER ? 4 : KL][NS];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t *p = kread + (in_ring + t * HALF) / 4, *ps = kscale + (in_ring + t * SHALF) / 4;
#pragma unroll
            for (int j = 0; j < KL; ++j) {
                if constexpr (KW == 4) {
                    const int4_t w = *reinterpret_cast<const int4_t *>(p + 256 * j);
#pragma unroll
                    for (int i = 0; i < 4; ++i) kd[t][j][i] = (uint32_t)w[i];
                } else {
                    const int2v_t w = *reinterpret_cast<const int2v_t *>(p + 128 * j);
                    kd[t][j][0] = (uint32_t)w[0];
                    kd[t][j][1] = (uint32_t)w[1];
                }
            }
            if constexpr (DEFER) {
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    const int4_t w = *reinterpret_cast<const int4_t *>(ps + 4 * i);
#pragma unroll
                    for (int e = 0; e < 4; ++e) (&ksd[t][0][0])[4 * i + e] = (uint32_t)w[e];
                }
            } else {
#pragma unroll
                for (int j = 0; j < KL; ++j) {
                    ksd[t][j][0] = ps[kgroup[j]];
                    if (32 * KW * j + 8 * KW * g >= a.D) ksd[t][j][0] = 0;
                }
            }
        }
        // the block after the next: its lookups, its keys in this one's place
        if constexpr (P16) {
            if (((n + 2) & 31) == 0) {
                look_up((n + 2) >> 5, nid);
                nid = table[key_page(a, key_of(place_of(((n + 2) >> 5) + 1)))];
            }
            gone[2] = dead >> (2 * ((n + 2) & 31)) & 3;
        } else {
            if ((n + 2) % ROWS4_IDS == 0) hold_ids(n + 2);
            if (n % 2 == 0) look_up((n + 2) / 2, ids[32 * ((n + 2) % ROWS4_IDS) + lane]);
            gone[2] = dead >> (32 * (n & 1)) & 0xffffffffu;
        }
        wait_reads();
        fetch_k(n + 2);

        float4_t s[QT][2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            if constexpr (DEFER) {
                float4_t acc[QT][NS];
#pragma unroll
                for (int ns = 0; ns < NS; ++ns) {
#pragma unroll
                    for (int qt = 0; qt < QT; ++qt) acc[qt][ns] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int w = 0; w < KW; ++w) {
                        const int4_t kf = places4(kd[t][ns][w]);
#pragma unroll
                        for (int qt = 0; qt < QT; ++qt) acc[qt][ns] = mfma_16(kf, q[qt][KW * ns + w], acc[qt][ns], f16_t());
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int ns = 0; ns < NS; ++ns) {
                        const half2_t sz = as_half2(ksd[t][i][ns]);
#pragma unroll
                        for (int qt = 0; qt < QT; ++qt) {
                            const float d = fmaf(-(float)sz[1], qsum[qt][ns], acc[qt][ns][i]);
                            s[qt][t][i] = fmaf(d, (float)sz[0], ns == 0 ? 0.f : s[qt][t][i]);      // (one instruction from fp16)
                        }
                    }
            } else {
#pragma unroll
                for (int qt = 0; qt < QT; ++qt) s[qt][t] = float4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int jl = 0; jl < KL; ++jl) {
                    const Zero z = zero_of(ksd[t][jl][0], ksd[t][jl][0]);
#pragma unroll
                    for (int w = 0; w < KW; ++w) {
                        const int4_t kf = values8(kd[t][jl][w], z);
#pragma unroll
                        for (int qt = 0; qt < QT; ++qt) s[qt][t] = mfma_16(kf, q[qt][KW * jl + w], s[qt][t], f16_t());
                    }
                }
            }
        }

        // loads of K n + 1, V n + 1 and K n + 2 stay on their way
        wait_loads<3 * FETCHES>();
        uint32_t vd[2][VC][VK], vsd[2][4][VC];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint8_t *p = vread + in_ring + t * HALF;
            const uint32_t *ps = vscale + (in_ring + t * SHALF) / 4;
#pragma unroll
            for (int x = 0; x < VC; ++x)
#pragma unroll
                for (int e = 0; e < VK; ++e) {
                    if constexpr (GM == 64)
                        vd[t][x][e] = *reinterpret_cast<const uint32_t *>(p + 256 * (2 * x + e));
                    else if constexpr (CH == 2)
                        vd[t][x][e] = *reinterpret_cast<const uint16_t *>(p + 128 * e);
                    else
                        vd[t][x][e] = *reinterpret_cast<const uint32_t *>(p + 1024 * x + 256 * e);
                }
            if constexpr (DEFER) {
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    const int4_t w = *reinterpret_cast<const int4_t *>(ps + 4 * i);
#pragma unroll
                    for (int e = 0; e < 4; ++e) (&vsd[t][0][0])[4 * i + e] = (uint32_t)w[e];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int x = 0; x < VC; ++x) vsd[t][i][x] = ps[i * n_s + vgroup[x]];
            }
        }
        wait_reads();
        fetch_v(n + 2);

        // a half needs a look at its keys where not every row sees all of them
        int key0[2];
        bool masked = gone[0] != 0 || v0 + 32 > end;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            key0[t] = key_at(kr, v0 + 16 * t);
            masked = masked || key0[t] + 16 > all_hi || (key0[t] < all_lo && key0[t] + 16 > a.sinks);
        }
        if (masked) {
            // (the comparisons stay in here)
            asm volatile("" : "+s"(key0[0]), "+s"(key0[1]));
            auto below = [](int n) { return (1 << min(max(n, 0), 4)) - 1; };       // bits of this lane's keys before the n-th
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int key = key0[t] + 4 * g;
                const int dead4 = P16 ? (gone[0] >> t & 1 ? 15 : 0) : (int)(gone[0] >> (16 * t + 4 * g)) & 15;
                const int open = below(end - v0 - 16 * t - 4 * g) & ~dead4, sinks = below(a.sinks - key);
                const int some = open & below(kr.hi - key) & (~below(kr.lo - key) | sinks);
                int mine[QT];
#pragma unroll
                for (int qt = 0; qt < QT; ++qt) mine[qt] = open & below(vhi[qt] - key) & (~below(vlo[qt] - key) | sinks);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int qt = 0; qt < QT; ++qt) {
                        const float was = s[qt][t][i];       // (a copy: bit_cast of a vector's element takes its first)
                        const int m = (mine[qt] << (31 - i)) >> 31;
                        s[qt][t][i] = __builtin_bit_cast(float, (__builtin_bit_cast(int, was) & m) | ((int)0xff800000u & ~m));
                    }
                    // values that no row sees may hold anything: they meet p = 0 as zeros
                    const uint32_t m = (uint32_t)((some << (31 - i)) >> 31);
#pragma unroll
                    for (int x = 0; x < VC; ++x) vsd[t][i][x] &= m;
                }
                if (!alike) {
                    bool any = false;
#pragma unroll
                    for (int e = 0; e < 4 * VC; ++e) any = any || is_nan(vsd[t][e / VC][e % VC]);
                    if (__any(any)) {       // such a value counts as 0, and is remembered
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int x = 0; x < VC; ++x) {
                                const bool nan = is_nan(vsd[t][i][x]);
                                const uint32_t at = DEFER ? (nan ? 0xffffu : 0u) : (uint32_t)(__ballot(nan) >> (16 * g)) & 0xffffu;
#pragma unroll
                                for (int qt = 0; qt < QT; ++qt) spoilt[qt] |= mine[qt] >> i & 1 ? at << (16 * x) : 0u;
                                vsd[t][i][x] = nan ? 0u : vsd[t][i][x];
                            }
                    }
                }
            }
        }
        gone[0] = gone[1];
        gone[1] = gone[2];
        float x[QT][8];
        int4_t p[QT];
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
            float mx = s[qt][0][0];
#pragma unroll
            for (int e = 1; e < 8; ++e) mx = fmaxf(mx, s[qt][e >> 2][e & 3]);
            mx *= sl[qt];
            if (__any(mx > m[qt] + A4_LAZY)) {         // also the first finite maximum: m is -inf
                mx = fmaxf(mx, __shfl_xor(mx, 16));
                mx = fmaxf(mx, __shfl_xor(mx, 32));
                float mn = fmaxf(m[qt], mx);
                if constexpr (DEFER) {
                    // the weights so far keep their places (and only their places: f is 1) up to the largest lift
                    mn = __builtin_floorf(mn);
#pragma unroll
                    for (int ns = 0; ns < NS; ++ns) {
                        const float was = lift[qt][ns];
                        lift[qt][ns] = fminf(was + (mn - m[qt]), A4_LIFT);      // (nothing seen: NaN, then the largest)
                        const float f = __builtin_amdgcn_exp2f(m[qt] - (mn == -INFINITY ? 0.f : mn) + (lift[qt][ns] - was));
                        if (n > 0) scale_group(qt, ns, f);
                        if (ns == 0) l[qt] *= f;
                    }
                    more[qt] = __builtin_amdgcn_exp2f(lift[qt][NS - 1] - lift[qt][0]);
                } else if (n > 0) {
                    const float al = __builtin_amdgcn_exp2f(m[qt] - (mn == -INFINITY ? 0.f : mn));
                    l[qt] *= al;
#pragma unroll
                    for (int xx = 0; xx < XT; ++xx) o[qt][xx] *= al;
                }
                m[qt] = mn;
            }
            const float base = (m[qt] == -INFINITY ? 0.f : m[qt]) - (DEFER ? TOP + lift[qt][0] : TOP);
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[qt][e] = __builtin_amdgcn_exp2f(fmaf(s[qt][e >> 2][e & 3], sl[qt], -base));
                sum += x[qt][e];
            }
            l[qt] += sum;
            if constexpr (!DEFER)
                p[qt] = int4_t{pack2(x[qt][0], x[qt][1], f16_t()), pack2(x[qt][2], x[qt][3], f16_t()), pack2(x[qt][4], x[qt][5], f16_t()),
                               pack2(x[qt][6], x[qt][7], f16_t())};
        }
        if constexpr (DEFER) {
#pragma unroll
            for (int ns = 0; ns < NS; ++ns) {
                int4_t zf;
#pragma unroll
                for (int y = 0; y < 4; ++y) zf[y] = (int)__builtin_amdgcn_perm(vsd[y >> 1][(2 * y & 3) + 1][ns], vsd[y >> 1][2 * y & 3][ns], 0x07060302u);
                auto weight = [&](int qt, int e) { return fmaf(ns == 0 ? x[qt][e] : x[qt][e] * more[qt], (float)as_half2(vsd[e >> 2][e & 3][ns])[0], 0.f); };
#pragma unroll
                for (int qt = 0; qt < QT; ++qt) {
                    half2_t top = half2_t{(f16_t)0.f, (f16_t)0.f};
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        p[qt][y] = pack2(weight(qt, 2 * y), weight(qt, 2 * y + 1), f16_t());
                        top = __builtin_elementwise_max(top, as_half2((uint32_t)p[qt][y]));
                    }
                    if (__any((float)__builtin_elementwise_max(top[0], top[1]) > 0x1p15f)) {      // (the first block's always)
                        float mine = 0.f;
#pragma unroll
                        for (int e = 0; e < 8; ++e) mine = fmaxf(mine, weight(qt, e));
                        mine = fmaxf(mine, __shfl_xor(mine, 16));
                        mine = fmaxf(mine, __shfl_xor(mine, 32));
                        const float by = fminf(TOP + 1.f - (float)__builtin_amdgcn_frexp_expf(mine), 0.f), f = __builtin_amdgcn_exp2f(by);
                        lift[qt][ns] += by;
                        if (n > 0) scale_group(qt, ns, f);
                        if (ns == 0) {
                            l[qt] *= f;
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[qt][e] *= f;
                        }
                        more[qt] = __builtin_amdgcn_exp2f(lift[qt][NS - 1] - lift[qt][0]);
#pragma unroll
                        for (int y = 0; y < 4; ++y) p[qt][y] = pack2(weight(qt, 2 * y), weight(qt, 2 * y + 1), f16_t());
                    }
                }
#pragma unroll
                for (int qt = 0; qt < QT; ++qt) oz[qt][ns] = mfma_16(zf, p[qt], oz[qt][ns], f16_t());
                // w[h][y]: elements 4h .. 4h + 3 of keys 2y and 2y + 1
                uint32_t w[VW / 4][4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    if constexpr (GM == 64) {
                        const uint32_t mine = vd[y >> 1][ns][y & 1], other = (uint32_t)__builtin_amdgcn_mov_dpp((int)mine, 0xb1, 0xf, 0xf, true);   // lane c ^ 1's
                        w[0][y] = __builtin_amdgcn_perm(mine, other, c & 1 ? 0x07060302u : 0x01000504u);
                    } else {
                        const uint32_t d0 = vd[y >> 1][ns][2 * y & 3], d1 = vd[y >> 1][ns][(2 * y & 3) + 1];
                        w[0][y] = __builtin_amdgcn_perm(d1, d0, 0x05040100u);
                        w[VW / 4 - 1][y] = __builtin_amdgcn_perm(d1, d0, 0x07060302u);
                    }
                }
#pragma unroll
                for (int h = 0; h < VW / 4; ++h)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        int4_t vf;
#pragma unroll
                        for (int y = 0; y < 4; ++y) vf[y] = places4(w[h][y])[e];
#pragma unroll
                        for (int qt = 0; qt < QT; ++qt) o[qt][VW * ns + 4 * h + e] = mfma_16(vf, p[qt], o[qt][VW * ns + 4 * h + e], f16_t());
                    }
            }
        } else {
#pragma unroll
            for (int xc = 0; xc < VC; ++xc) {
                Zero z[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) z[y] = zero_of(vsd[y >> 1][2 * y & 3][xc], vsd[y >> 1][(2 * y & 3) + 1][xc]);
#pragma unroll
                for (int h = 0; h < VW / 4; ++h) {
                    uint32_t w[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y) w[y] = __builtin_amdgcn_perm(vd[y >> 1][xc][(2 * y & 3) + 1], vd[y >> 1][xc][2 * y & 3], h ? 0x07060302u : 0x05040100u);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        int4_t vf;
#pragma unroll
                        for (int y = 0; y < 4; ++y) vf[y] = e & 1 ? value2<true>(e & 2 ? w[y] >> 8 : w[y], z[y]) : value2<false>(e & 2 ? w[y] >> 8 : w[y], z[y]);
#pragma unroll
                        for (int qt = 0; qt < QT; ++qt) o[qt][VW * xc + 4 * h + e] = mfma_16(vf, p[qt], o[qt][VW * xc + 4 * h + e], f16_t());
                    }
                }
            }
        }
    }
    if constexpr (DEFER) {      // the codes' places, scales and zero-points
#pragma unroll
        for (int qt = 0; qt < QT; ++qt)
#pragma unroll
            for (int x = 0; x < XT; ++x) {
                const float f = (x & 1 ? 0x1p18f : 0x1p22f);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    o[qt][x][i] = fmaf(o[qt][x][i], f, -oz[qt][x / VW][0]);
                    if (x / VW > 0) o[qt][x][i] *= 1.f / more[qt];      // (a power of two)
                }
            }
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) m[qt] -= lift[qt][0];
    }

#pragma unroll
    for (int qt = 0; qt < QT; ++qt) {
        if (!__any(spoilt[qt] != 0)) continue;
        spoilt[qt] |= __shfl_xor(spoilt[qt], 16);
        spoilt[qt] |= __shfl_xor(spoilt[qt], 32);
#pragma unroll
        for (int x = 0; x < XT; ++x)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[qt][x][i] = spoilt[qt] >> (16 * (x / VW) + 4 * g + i) & 1 ? NAN : o[qt][x][i];
    }

    // the ring is done with: nothing is on its way into LDS any more, from no wave
    wait_loads<0>();
    __syncthreads();
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
        const int r = rb * a.rows + row, i = a.by_g(r), hq = hk * a.g + (r - i * a.g);
        const int64_t t = kr.t0 + i;
        // no sum: no key, or scores of -inf by overflow (of a split: the join looks)
        const bool none = tot == 0.f && (a.splits > 1 || !row_sees(a, b, kr, i));
        const float inv = 1.f / (tot > 0.f ? tot : NAN);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = none ? 0.f : sum[e] * inv;
        const float lse2 = none ? -INFINITY : mm - TOP + __builtin_amdgcn_logf(tot > 0.f ? tot : NAN);
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
// The matrix instructions and the softmax between them bound it, which share a SIMD's issue: 2 prompts of 4096
// tokens, 32 heads of 128: 321 to 338 us (cards differ), 814 to 857 TFLOP/s of a large product's 1216, matrix instructions in 39 % of the
// cycles and vector ones in 54 %.  Taking the codes out costs what reading rows of 16 bits does (those: 335
// us).  Masks as a bit a key (compared key by key 337 on the card of 326; 16 chunks of up to 256 tokens 37.6, now 34.3).  D = 256
// has one wave a SIMD (2 chunks of 300 on up to 8192 keys, 16 heads: 234 us, 275 TFLOP/s).
// Values of NaN: rows that do not see them get 0 times NaN too, so a workgroup whose outputs hold NaN goes again, with
// such values as 0 and a look at each tile's scales for who sees them.  (Looking in the first pass would cost every tile.)
// ---------------------------------------------------------------------------
__host__ __device__ constexpr int tiles4_keys(int D) { return D <= 128 ? 64 : 32; }
__host__ __device__ constexpr int tiles4_waves(int D) { return D <= 128 ? 8 : 4; }

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

    const int above = a.by_groups(blockIdx.x), bh = blockIdx.x - above * a.by_groups.d;     // sequence and head fastest: one head's blocks share an L2
    const int top = above / a.splits, split = above - top * a.splits, rb = a.rblocks - 1 - top;   // the longest blocks first
    const int b = a.by_Hkv(bh), hk = bh - b * a.Hkv;

    const Range4 kr = range4(a, b, rb);
    const int nrow = min(32 * NW, kr.n * a.g - rb * a.rows);
    if (nrow <= 0) return;
    const int begin = split * a.chunk, end = min(kr.len, begin + a.chunk);
    if (begin >= end && split > 0) return;

    const int tid = threadIdx.x, lane = tid & 63, wave = wave_id(), c = lane & 31, h = lane >> 5;
    const S tag = (S)0.f;

    // this lane's row
    const int r = rb * a.rows + 32 * wave + c, i = a.by_g(r), hq = hk * a.g + (r - i * a.g);
    const bool live = 32 * wave + c < nrow;
    const int vhi = live ? kr.L - kr.n + i + 1 : 0, vlo = a.window > 0 ? vhi - a.window : 0;
    int4_t q[QJ];
    float sl = a.scale * ATT_LOG2E;
    {
        const char *row = (const char *)a.q + (int64_t)(kr.t0 + (live ? i : 0)) * a.q_ts + (int64_t)(live ? hq : 0) * a.q_hs;
        uint32_t bits = 0;
#pragma unroll
        for (int j = 0; j < QJ; ++j) {
            const int d = 16 * j + 8 * h;
            q[j] = *reinterpret_cast<const int4_t *>(row + (d < a.D ? 2 * d : 0));
            if (!live || d >= a.D) q[j] = int4_t{0, 0, 0, 0};
            if constexpr (!__is_same(S, f16_t)) bits = larger2(bits, q[j]);
        }
#pragma unroll
        for (int j = 0; j < QJ; ++j) q[j] = code_order(q[j]);
        if constexpr (!__is_same(S, f16_t)) {
            const float top = size_of(max(bits & 0xffffu, bits >> 16), tag);
            const int up = rise_of(fmaxf(top, __shfl_xor(top, 32)));
            scale_row<false, QJ>(q, up, tag);
            sl = fminf(ldexpf(sl, -up), 3e38f);
        }
        sl = above_zero(sl);
    }
    // keys that some row of the wave sees, and keys that all of them see
    const int wr0 = rb * a.rows + 32 * wave, wr1 = min(wr0 + 31, rb * a.rows + nrow - 1);
    const bool wlive = 32 * wave < nrow;
    const int whi = wlive ? kr.L - kr.n + a.by_g(wr1) + 1 : 0, wall_hi = wlive ? kr.L - kr.n + a.by_g(wr0) + 1 : 0;
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
    int *again = reinterpret_cast<int *>(masks + SLOTS);
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
    const uint8_t *kb = kbase + in_row, *vb = vbase + in_row, *ksb = ksbase + in_scales, *vsb = vsbase + in_scales;
    auto load_tile = [&](int tile) {
        const int slot = tile % SLOTS;
        const int4_t mk = masks[slot];
#pragma unroll
        for (int n = 0; n < LN; ++n) {
            const int4_t at = places[2 * (slot * KB + srow + SSTEP * n)], as = places[2 * (slot * KB + srow + SSTEP * n) + 1];
            kst[n] = *reinterpret_cast<const uint32_t *>(kb + off64(at[0], at[1]));
            vst[n] = *reinterpret_cast<const uint32_t *>(vb + off64(at[2], at[3]));
            kss[n] = *reinterpret_cast<const uint32_t *>(ksb + off64(as[0], as[1]));
            vss[n] = *reinterpret_cast<const uint32_t *>(vsb + off64(as[2], as[3]));
        }
        vlive = uniform64(mk[0], mk[1]);
        hidden = uniform64(mk[2], mk[3]);
    };
    uint64_t careful = 0;         // uniform, 0 or 1
    auto store_tile = [&](int buf) {
        if (~vlive | careful) {     // what no row sees may hold anything: it meets p = 0 as zeros
#pragma unroll
            for (int n = 0; n < LN; ++n) vss[n] = (vlive >> (srow + SSTEP * n)) & 1 && !(careful && is_nan(vss[n])) ? vss[n] : 0;
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

    float m, l;
    float16v_t o[XT];
    uint32_t spoilt = 0;          // groups in which this lane's row sees a value of NaN
    const int tiles = (max(0, end - begin) + KB - 1) / KB;
    if (tid == 0) *again = 0;
anew:
    m = -INFINITY, l = 0.f;
#pragma unroll
    for (int x = 0; x < XT; ++x)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[x][e] = 0.f;
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
            if (v0 + KB > end || key0 + KB > wall_hi || (key0 < wall_lo && key0 + KB > kr.sk) || (bad | careful)) {
                // element e of tile t is key key0 + 4 h + 32 t + e % 4 + 8 (e / 4) (v0 + KB > end with the last places alone: key >= vhi there)
                const int to = min(vhi, key0 + end - v0) - key0 - 4 * h, from = vlo - key0 - 4 * h, sinks = kr.sk - key0 - 4 * h;
                auto below = [](int n) { return n >= 64 ? ~uint64_t(0) : (uint64_t(1) << max(n, 0)) - 1; };      // keys before the n-th
                const uint64_t mine = below(to) & (~below(from) | below(sinks)) & ~(bad >> (4 * h));
                if (careful) {       // lane l: the scales of key l's values
                    const int4_t as = places[2 * (tile % SLOTS * KB + (lane & (KB - 1))) + 1];
                    for (int e = 0; e < a.D >> a.lg_G; ++e) {
                        const uint64_t nan = __ballot(is_nan(*reinterpret_cast<const uint32_t *>(vsbase + off64(as[2], as[3]) + 4 * e)));
                        spoilt |= ((KB == 64 ? nan : nan & 0xffffffffu) >> (4 * h) & mine) != 0 ? 1u << e : 0u;
                    }
                }
                const int word[2] = {(int)(uint32_t)mine, (int)(uint32_t)(mine >> 32)};
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const int m = (word[t] << (31 - (e & 3) - 8 * (e >> 2))) >> 31;
                        const float was = s[t][e];       // (a copy: bit_cast of a vector's element takes its first)
                        s[t][e] = __builtin_bit_cast(float, (__builtin_bit_cast(int, was) & m) | ((int)0xff800000u & ~m));
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

    // A value of NaN has reached every row of its block, also those that do not see it: once more, with such values as 0
    // and with a note of who sees them.
    if (!careful) {
        float all = 0.f;
#pragma unroll
        for (int x = 0; x < XT; ++x)
#pragma unroll
            for (int e = 0; e < 16; ++e) all += o[x][e];
        if (__any(all != all && l == l) && lane == 0) *again = 1;
        __syncthreads();
        if (*again) {
            careful = 1;
            goto anew;
        }
    }

    l += __shfl_xor(l, 32);
    spoilt |= __shfl_xor(spoilt, 32);
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
            for (int k = 0; k < 4; ++k) y[k] = none ? 0.f : spoilt >> (d >> a.lg_G) & 1 ? NAN : o[x][e + k] * inv;
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
    const int rb = (min(i, a.max_q - 1) * a.g + hq - a.by_g(hq) * a.g) / a.rows;
    const Range4 kr = range4(a, b, rb);
    const bool live = i < a.max_q && i < kr.n;
    if (JW == 4 && !live) return;                    // the whole workgroup
    const int splits = live ? max(1, (kr.len + a.chunk - 1) / a.chunk) : 0;
    const int64_t row = live ? (int64_t)(kr.t0 + i) * a.Hq + hq : 0;
    const float *lses = a.part + (int64_t)a.T * a.Hq * a.splits * a.D + row * a.splits;
    const int d = 4 * (lane % LN);
    const float *part = a.part + row * a.splits * a.D + (d < a.D ? d : 0);
    // the first four of a lane's splits are on their way before the maximum is known
    constexpr int AHEAD = 4, STEP = JW * SW;
    const int s0 = part_wave * SW + lane / LN;
    float4_t o[AHEAD];
    float lse[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
        const int s = max(0, min(s0 + k * STEP, splits - 1));
        lse[k] = lses[s];
        o[k] = *reinterpret_cast<const float4_t *>(part + (int64_t)s * a.D);
    }
    float mm = -INFINITY;
    for (int s = lane; s < splits; s += 64) mm = fmaxf(mm, lses[s]);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) mm = fmaxf(mm, __shfl_xor(mm, x));
    const float ms = mm == -INFINITY ? 0.f : mm;
    float4_t sum = float4_t{0.f, 0.f, 0.f, 0.f};
    float tot = 0.f;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
        if (s0 + k * STEP < splits) {
            const float f = __builtin_amdgcn_exp2f(lse[k] - ms);
            tot += f;
            sum += f * o[k];
        }
#pragma unroll 4
    for (int s = s0 + AHEAD * STEP; s < splits; s += STEP) {
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

int64_t plan_attend4(Attend4Args &a)
{
    Divisor by_page;
    by_page.set(a.page);
    a.page_mul = by_page.mul, a.page_sh = by_page.sh;

    const int64_t rows = (int64_t)a.max_q * a.g;
    const bool tiles = rows > 32;
    a.rows = tiles ? 32 * tiles4_waves(a.D) : rows <= 16 || a.D > 128 ? 16 : 32;
    a.rblocks = (int)((rows + a.rows - 1) / a.rows);
    a.lg_unit = !tiles ? 4 : tiles4_keys(a.D) == 64 ? 6 : 5;
    int64_t span = a.max_kv;
    if (a.window > 0)
        span = std::min(span, (int64_t)a.window + (a.rows + a.g - 1) / a.g + (((std::min(a.sinks, a.max_kv) - 1) >> a.lg_unit) + 1 << a.lg_unit));
    span += 15;
    const int64_t heads = (int64_t)a.B * a.Hkv, groups = heads * a.rblocks;
    if (heads < (int64_t(1) << 31)) a.by_groups.set(heads);        // (more are refused)
    a.by_Hkv.set(a.Hkv);
    a.by_rblocks.set(a.rblocks);
    a.by_g.set(a.g);
    int64_t splits, unit;
    if (tiles) {
        // One workgroup a CU, 256 at once: what counts is in how many rounds the blocks of rows go, and what
        // shares of their keys cost, fp32 sums for each output written and read.  A share takes about
        // (12 + D / 5) ns a key and 5 us; of the shares that fill r rounds the largest number is the
        // quickest.  (us: 3 x up to 600 tokens, 8 heads of 4, a window of 4096: 159 whole, 191 in two
        // shares; one chunk of 600 on 32768 keys: 1035 whole, 379 in three, 562 in four; 50 tokens on
        // 48752 keys, one head of 2: 25 in 152, 70 in 19; 15 x 124 tokens on up to 3078 keys, 4 heads: 79
        // whole, 40 in four; 4 x 512 on 2048: 77 and 128 in two.)
        unit = 128;
        const int64_t live = std::min(groups, a.Hkv * (((int64_t)a.T * a.g + a.rows - 1) / a.rows + a.B / 2));     // blocks with rows
        const double key = (12.0 + a.D / 5.0) * 1e-3, share = 8.0 * a.T * a.Hq * (a.D + 1) / 4.5e6;
        auto cost = [&](int64_t s) { return (double)((live * s + 255) / 256) * ((double)span / s * key + 5.0) + (s > 1 ? 5.0 + share * s : 0.0); };
        splits = 1;
        for (int64_t round = 1; round <= 4; ++round) {
            const int64_t s = std::min(256 * round / std::max<int64_t>(1, live), span / unit);
            if (s > 1 && cost(s) < cost(splits)) splits = s;
        }
    } else {
        // The GPU holds 1024 workgroups at once; with at least 64 KB of codes and scales each, or 16 KB
        // where there are few (4 sequences of up to 131071 keys, 8 heads, us: 96 in 24 shares, 97 in 32, 98
        // in 48; one of 5000, G 64: 19.5 in 4, 13.8 in 16, 12.8 in 32).  Many sequences are hardly ever alike in
        // length: shares of 160 KB let the GPU even them out (64 of up to 8192, G 128: 65 in 4, 77 in 2).  One
        // launch without a join is enough where the keys are few.
        unit = 32 * rows4_waves(a.D);
        const int64_t bytes = (span - 15) * (a.D + 8 * (a.D >> a.lg_G)), kb = 1024;
        splits = std::max(std::min(256 / groups, (bytes + 16 * kb - 1) / (16 * kb)),
                          std::max<int64_t>(1, std::min((1024 + groups - 1) / groups, (bytes + 64 * kb - 1) / (64 * kb))));
        if (groups >= 128) splits = std::max(splits, std::min((2048 + groups - 1) / groups, bytes / (160 * kb)));
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
    const size_t lds = (size_t)4 * KB * DP * 2 + 2 * NW * (2 * KB + 1) * 16 + 16;   // tiles, places, masks, whether to go again
    const hipError_t e = allow_lds(&attend4_tiles_kernel<S, DC, NW>, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((attend4_tiles_kernel<S, DC, NW>), dim3((unsigned)((int64_t)a.B * a.rblocks * a.Hkv * a.splits)), dim3(64 * NW), lds, st, a);
    return hipGetLastError();
}

template <typename S, int DP, int GM, int PAGES, int QT>
static hipError_t rows4_go(const Attend4Args &a, hipStream_t st)
{
    constexpr int NW = rows4_waves(DP);
    const int nrow = (int)std::min<int64_t>(16 * QT, (int64_t)a.max_q * a.g);
    const size_t lds = std::max<size_t>((size_t)NW * nrow * (DP + 6) * 4, NW * rows4_ring(DP, GM, PAGES));   // join, ring
    const hipError_t e = allow_lds(&attend4_rows_kernel<S, DP, GM, PAGES, QT>, lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((attend4_rows_kernel<S, DP, GM, PAGES, QT>), dim3((unsigned)((int64_t)a.B * a.rblocks * a.Hkv * a.splits)), dim3(64 * NW), lds, st, a);
    return hipGetLastError();
}

template <typename S, int DP, int GM, int PAGES>
static hipError_t rows4_pick(const Attend4Args &a, hipStream_t st)
{
    if constexpr (DP <= 128) {
        if (a.rows == 32) return rows4_go<S, DP, GM, PAGES, 2>(a, st);
    }
    return rows4_go<S, DP, GM, PAGES, 1>(a, st);
}
// Groups that leave the codes as they are where they pay: of 64 in rows of 64 and 128, of 128 in rows of 128
// and 256 (64 users of up to 8192 keys, us, so and as (c - z) s: D 64, G 64: 49 and 57; D 128, G 128: 64 and 73, two tiles of rows
// 98 and 104; D 128, G 64: 76 and 80, pages of 100 tokens 79 and 83; D 256, G 128, up to 4096 keys: 83 and 92).  Two tiles of rows
// with groups of 64 in rows of 128 have not the registers for it (105 and 102).
template <typename S, int DP, int PAGES>
static hipError_t rows4_by_group(const Attend4Args &a, hipStream_t st)
{
    constexpr int GM = DP == 64 ? 64 : 128;
    if (a.D == DP && (1 << a.lg_G) == GM) return rows4_pick<S, DP, GM, PAGES>(a, st);
    if constexpr (DP == 128) {
        if (a.D == DP && a.lg_G == 6 && a.rows == 16) return rows4_go<S, DP, 64, PAGES, 1>(a, st);
    }
    return rows4_pick<S, DP, 32, PAGES>(a, st);
}

// SHARED: what a page holds of a head is a cache line at most, and neighbouring heads read the same lines (64 users
// of up to 8192 keys, us, so and as any page: D 128, pages of 1 token 125 and 188, of 2 96 and 110, of 4 89 and 86;
// D 32, of 1 96 and 208, of 8 95 and 97; D 256, up to 4096, of 1 126 and 147, of 2 122 and 117).
template <typename S, int DP>
static hipError_t rows4_by_pages(const Attend4Args &a, hipStream_t st)
{
    if (a.halves) return rows4_by_group<S, DP, HALVES>(a, st);
    return a.page * a.D / 2 <= 128 ? rows4_by_group<S, DP, SHARED>(a, st) : rows4_by_group<S, DP, ANY>(a, st);
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
        e = rows4_by_pages<S, 64>(a, st);
    else if (a.D <= 128)
        e = rows4_by_pages<S, 128>(a, st);
    else
        e = rows4_by_pages<S, 256>(a, st);
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
    const int64_t threads = 64 * (a.rows > 32 ? tiles4_waves(a.D) : rows4_waves(a.D));
    if (groups > most || a.rblocks * groups > most / threads / a.splits) return false;
    return a.splits == 1 || join4_blocks(a) <= most / 256 / a.B;
}

hipError_t launch_attend4(const Attend4Args &a, bool bf16, hipStream_t st)
{
    if (!attend4_fits(a)) return hipErrorNotSupported;
    return bf16 ? attend4_type<bf16_t>(a, st) : attend4_type<f16_t>(a, st);
}

}  // namespace qmm
