// stream.hip -- qmm_linear for 2 to 64 rows of X: the weights are streamed once
// and every run is dequantised once for all rows.
//
// Bound by the packed weights' bytes; next to that by the unpacking (about 50
// VALU operations for a lane's 32 codes at 4 bits).  A workgroup of W waves takes
// a slice of K and stages X's slice in LDS once, in the unpack's slot order; its
// waves then take a 16-column tile each, walk the slice with STREAM_D steps of
// 128 rows of weights in flight, and hold the tile's sums alone: no sum over
// waves.  In a step lane group g owns run 4t + g of column lane % 16, as in the
// other MFMA kernels, and w = (q - z) s as there: q - z exact in fp16, one
// rounding by s; each dequantised run meets the RB blocks of 16 rows in turn.
// Where there is more than one slice the sums go to the workspace in fp32 and
// stream_join_kernel adds the slices in order and applies the epilogue.
// Measured at K 28672, N 8192, 4 bits, G 128 with zero-points, 16 rows: 27 us (and 4.6
// for the join) where the weights come from the last-level cache, 38.9 a call with
// weights from HBM, 3.2 TB/s; without the unpacking 23.5, without X too 22.7, 2 steps in
// flight instead of 4: 30.9.  16 waves hold the whole column tiles of a CU's share; K
// split over the waves of a workgroup instead (X fragments in registers, sums joined in
// LDS) took 81.
#define QMM_EPILOGUE
#include <algorithm>

#include "launch.hpp"
#include "qmm_device.hpp"
#include "epilogue.hpp"

namespace qmm {

constexpr uint32_t STREAM_OOB = 0x80000000u;
constexpr int STREAM_D = 4;        // steps of weights in flight
constexpr int STREAM_LDS = 128 * 1024;

// most waves of a workgroup: 16 leave 128 registers a wave, which more row blocks overrun
__host__ __device__ constexpr int stream_waves(int RB) { return RB > 1 ? 8 : 16; }

// X in LDS: [run][row] of 64 bytes, the 16-byte chunks XOR-ed with the run and the
// row as in the GEMM's tiles: no bank conflicts in the fragment reads
__device__ __forceinline__ int stream_chunk(int row, int run, int q) { return 16 * (q ^ ((3 * run) & 3) ^ ((row >> 2) & 3)); }

template <int BITS, bool PGZ, int RB, bool G128>
__global__ __launch_bounds__(64 * stream_waves(RB)) void stream_kernel(const uint16_t *__restrict__ X, const uint32_t *__restrict__ wq,
                                                        const uint16_t *__restrict__ s, const uint16_t *__restrict__ z,
                                                        uint16_t *__restrict__ Y, float *__restrict__ part, int M, int K, int N, int G,
                                                        int steps, const Epilogue ep)
{
    using P = RunPlan<BITS>;
    constexpr int D = STREAM_D, ROWS = 16 * RB;
    // Where a step is one group its sum can be scaled in fp32 instead of its weights in
    // fp16: 4 RB operations for 16.
    constexpr bool AFTER = G128 && RB <= 2;
    extern __shared__ __attribute__((aligned(16))) uint8_t xs[];   // [4 steps][ROWS] of 64 bytes
    const int tid = threadIdx.x, lane = tid & 63, wave = wave_id(), g = lane >> 4, c = lane & 15;
    const int R = K >> 5, ng = K / G, tiles = (N + 15) >> 4;
    const float ginv = run_group_inv(G);
    const uint32_t run_bytes = 4u * BITS, col_bytes = (uint32_t)R * run_bytes;
    const int run0 = (int)blockIdx.y * steps * 4, run1 = min(R, run0 + 4 * steps);   // the slice (steps: a multiple of D)
    const float zdef = (float)(1u << (BITS - 1));

    uint32_t d[D][BITS];
    // step st of a tile into ring slot i; tiles and runs that are not there load zeros
    auto issue = [&](int tile, int st, int i) {
        const int t = min(tile, tiles - 1), cols = tile < tiles ? min(16, N - 16 * t) : 0;
        const __amdgpu_buffer_rsrc_t wr = make_rsrc(wq + (size_t)t * 16 * R * BITS, (uint32_t)cols * col_bytes);
        const int run = run0 + 4 * st + g;
        load_dwords<LOAD_DEFAULT>(wr, run < run1 ? (uint32_t)c * col_bytes + (uint32_t)run * run_bytes : STREAM_OOB, d[i], BITS);
    };
    // s and z of the D steps from st on: 16 runs, so at most 16 groups from that of the
    // first run on.  G128 (G = 128): step and group are one, and every lane loads its
    // column's four; else lane group g loads groups 4g .. 4g + 3 and the lanes
    // take theirs from each other (a 2-byte load for each step and lane costs more
    // requests than the weights: 46 -> 63 us for K 28672, N 8192, 16 rows with the
    // zero-points loaded so).  Loads are dwords: the three that hold four halves.
    uint32_t sw[3], zw[3];
    auto first_group = [&](int st) { return G128 ? (run0 >> 2) + st : run_group(min(run0 + 4 * st, R - 1), ginv); };
    auto issue_sz = [&](int tile, int st) {
        const int t = min(tile, tiles - 1), cols = tile < tiles ? min(16, N - 16 * t) : 0;
        const uint32_t bytes = ((uint32_t)(cols * ng) * 2u + 3u) & ~3u;
        const int at = c * ng + first_group(st) + (G128 ? 0 : 4 * g);
        load_dwords<LOAD_DEFAULT>(make_rsrc(s + (size_t)t * 16 * ng, bytes), (uint32_t)(at >> 1) * 4u, sw, 3);
        if constexpr (PGZ) load_dwords<LOAD_DEFAULT>(make_rsrc(z + (size_t)t * 16 * ng, bytes), (uint32_t)(at >> 1) * 4u, zw, 3);
    };
    auto four = [&](const uint32_t (&w)[3], int st, uint16_t (&v)[D]) {
        const int first = first_group(st);
        const bool odd = (c * ng + first + (G128 ? 0 : 4 * g)) & 1;
        uint32_t lo = odd ? __builtin_amdgcn_alignbit(w[1], w[0], 16) : w[0];
        uint32_t hi = odd ? __builtin_amdgcn_alignbit(w[2], w[1], 16) : w[1];
        if constexpr (G128) {
            // past the slice's last step stand the next column's, which may be no numbers
            const int left = (run1 - run0) / 4 - st;
            lo &= left >= 2 ? 0xffffffffu : left == 1 ? 0xffffu : 0u;
            hi &= left >= 4 ? 0xffffffffu : left == 3 ? 0xffffu : 0u;
        }
#pragma unroll
        for (int i = 0; i < D; ++i) {
            if constexpr (G128) {
                v[i] = (uint16_t)((i & 2 ? hi : lo) >> (16 * (i & 1)));
            } else {
                const int k = run_group(min(run0 + 4 * (st + i) + g, R - 1), ginv) - first, src = 16 * (k >> 2) + c;
                const uint32_t x = (uint32_t)__shfl((int)lo, src), y = (uint32_t)__shfl((int)hi, src);
                v[i] = (uint16_t)((k & 2 ? y : x) >> (16 * (k & 1)));
            }
        }
    };
    const int W = (int)blockDim.x >> 6;
    const int stride = (int)gridDim.x * W;
    int tile = (int)blockIdx.x * W + wave;
#pragma unroll
    for (int i = 0; i < D; ++i) issue(tile, i, i);
    issue_sz(tile, 0);

    // stage X's slice: (run, row) pieces, runs fastest, zeros past M and past the slice
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(X, (uint32_t)(M * K * 2));
    for (int it = tid; it < 4 * steps * ROWS; it += 64 * W) {
        const int row = it / (4 * steps), r = it - row * 4 * steps;
        uint32_t raw[16];
        load_dwords<LOAD_DEFAULT>(xr, (run0 + r < run1 && row < M) ? ((uint32_t)row * K + (uint32_t)(run0 + r) * 32u) * 2u : STREAM_OOB, raw, 16);
        _Float16 x[32];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const half2_t p = as_half2(raw[i]);
            x[2 * i] = p[0];
            x[2 * i + 1] = p[1];
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            half8_t v;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = x[P::code[8 * q + e]];
            *reinterpret_cast<half8_t *>(xs + (size_t)(r * ROWS + row) * 64 + stream_chunk(row, r, q)) = v;
        }
    }
    __syncthreads();
    const uint8_t *xa[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) xa[u] = xs + (g * ROWS + c) * 64 + stream_chunk(c, g, u);

    for (; tile < tiles; tile += stride) {
        float4_t acc[RB];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) acc[rb] = float4_t{0.f, 0.f, 0.f, 0.f};
        for (int s0 = 0; s0 < steps; s0 += D) {
            uint16_t sv[D], zv[D];
            four(sw, s0, sv);
            if constexpr (PGZ) four(zw, s0, zv);
            if (s0 + D < steps)
                issue_sz(tile, s0 + D);
            else
                issue_sz(tile + stride, 0);
#pragma unroll
            for (int i = 0; i < D; ++i) {
                uint32_t h[16];
                run_to_half2<BITS>(d[i], h);
                half2_t s2, z2;
                s2[0] = s2[1] = as_half(sv[i]);
                z2[0] = z2[1] = as_half(PGZ ? zv[i] : (uint16_t)0);
                half8_t w8[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = 4 * u + e;
                        half2_t pinv, base;
                        pinv[0] = (_Float16)pow2neg(P::pos[2 * j]);
                        pinv[1] = (_Float16)pow2neg(P::pos[2 * j + 1]);
                        base[0] = (_Float16)(1024.0f * pow2neg(P::pos[2 * j]) + (PGZ ? 0.0f : zdef));
                        base[1] = (_Float16)(1024.0f * pow2neg(P::pos[2 * j + 1]) + (PGZ ? 0.0f : zdef));
                        if (PGZ) base = base + z2;
                        half2_t w = as_half2(h[j]) * pinv - base;
                        if constexpr (!AFTER) w = w * s2;
                        w8[u][2 * e] = w[0];
                        w8[u][2 * e + 1] = w[1];
                    }
                // the slot is free: the step D ahead, of this tile or the wave's next one
                if (s0 + D < steps)
                    issue(tile, s0 + D + i, i);
                else
                    issue(tile + stride, i, i);
                float4_t y[RB];
#pragma unroll
                for (int rb = 0; rb < RB; ++rb) y[rb] = AFTER ? float4_t{0.f, 0.f, 0.f, 0.f} : acc[rb];
#pragma unroll
                for (int u = 0; u < 4; ++u)
#pragma unroll
                    for (int rb = 0; rb < RB; ++rb) {
                        const half8_t x8 = *reinterpret_cast<const half8_t *>(xa[u] + (4 * (s0 + i) * ROWS + 16 * rb) * 64);
                        y[rb] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x8, w8[u], y[rb], 0, 0, 0);
                    }
#pragma unroll
                for (int rb = 0; rb < RB; ++rb)
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[rb][k] = AFTER ? fmaf((float)s2[0], y[rb][k], acc[rb][k]) : y[rb][k];
            }
        }
        // lane (g, c) holds rows 4g .. 4g + 3 of column c
        const int col = 16 * tile + c;
        if (col < N) {
#pragma unroll
            for (int rb = 0; rb < RB; ++rb)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 16 * rb + 4 * g + i;
                    if (row >= M) continue;
                    if (part)
                        part[((size_t)blockIdx.y * M + row) * N + col] = acc[rb][i];
                    else
                        Y[(size_t)row * N + col] = f32_to_f16_bits(epilogue_at(ep, acc[rb][i], row, col, N));
                }
        }
    }
}

// the slices' sums, added in order, and the epilogue; V columns a thread
template <int V>
__global__ __launch_bounds__(256) void stream_join_kernel(const float *__restrict__ part, uint16_t *__restrict__ Y, int slices, int M,
                                                          int N, const Epilogue ep)
{
    const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V, MN = (int64_t)M * N;
    if (at >= MN) return;
    float h[V];
#pragma unroll
    for (int e = 0; e < V; ++e) h[e] = 0.f;
#pragma unroll 8
    for (int p = 0; p < slices; ++p) {
        if constexpr (V == 4) {
            const float4_t x = *reinterpret_cast<const float4_t *>(part + p * MN + at);
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] += x[e];
        } else {
            h[0] += part[p * MN + at];
        }
    }
    const int row = (int)(at / N), col = (int)(at - (int64_t)row * N);
#pragma unroll
    for (int e = 0; e < V; ++e) Y[at + e] = f32_to_f16_bits(epilogue_at(ep, h[e], row, col + e, N));
}

hipError_t launch_join(const GemvArgs &a, const float *part, int slices, hipStream_t st)
{
    const int64_t n = (int64_t)a.M * a.N;
    if (a.N % 4 == 0)
        hipLaunchKernelGGL((stream_join_kernel<4>), dim3((unsigned)((n / 4 + 255) / 256)), dim3(256), 0, st, part, a.Y, slices, a.M, a.N, a.ep);
    else
        hipLaunchKernelGGL((stream_join_kernel<1>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, part, a.Y, slices, a.M, a.N, a.ep);
    return hipGetLastError();
}

struct StreamPlan {
    int RB, W, steps, slices, groups;
};
static StreamPlan stream_plan(int M, int K, int N)
{
    StreamPlan p;
    p.RB = M <= 16 ? 1 : M <= 32 ? 2 : 4;
    const int all = (K / 32 + 3) / 4, tiles = (N + 15) / 16, most = STREAM_LDS / (64 * 64 * p.RB);
    p.W = std::min(stream_waves(p.RB), tiles >= 512 ? 16 : 8);
    const int groups = (tiles + p.W - 1) / p.W;
    // one workgroup a CU where columns and slices can give them
    const int slices = std::max(1, std::max((all + most - 1) / most, std::min(256 / groups, all / 4)));
    p.steps = ((all + slices - 1) / slices + STREAM_D - 1) / STREAM_D * STREAM_D;
    p.slices = (all + p.steps - 1) / p.steps;
    p.groups = std::min(groups, std::max(1, 512 / p.slices));
    return p;
}

bool stream_takes(int M, int K, int N)
{
    // Up to 16 rows the GEMV kernels hold X's fragments in registers and need no join up
    // to K = 8192; beyond, they take K in passes (K 28672, N 8192, 16 rows, 4 bits: 60 us,
    // here 39).  From 17 on the GEMM's smallest tiles leave CUs idle or dequantise every
    // weight again for each tile of rows; it is quicker for small products alone, where
    // the join's launch counts.  The GEMM and here, 4 bits, us:
    //   K x N            17 rows      32           33           64
    //   2048 x 4096    6.8   9.1   7.7   9.7   12.6  10.4   13.6  11.4
    //   4096 x 3000   11.2   9.0  10.9   9.6   13.5  10.6   18.0  12.5
    //   4096 x 4096   11.4   9.5  11.1  10.3   13.4  11.4   18.1  14.3
    //   8192 x 2048   11.7   9.5  13.5  10.7   13.9  12.0   19.6  14.5
    //   2048 x 8192   10.1   9.9  10.3  10.9   11.1  12.1   12.2  14.4
    //   4096 x 6000   14.7  10.9  16.4  11.9   16.6  14.0   20.7  15.6
    //   4096 x 11008  22.2  13.4  22.6  14.1   22.9  22.4   26.9  24.5
    // K N = 14M parts these but for the second row and, by up to a fifth, for long rows of
    // few steps (K 2048, N 8192) and 33 rows and more of the first; 2 and 8 bits lie alike.
    // A few columns of long K are one or two workgroups' work for either of them (16 rows,
    // K 7808, N 2: 14.8 us, in slices 9.3).
    if (M < 2 || M > 64) return false;
    if (!(K >= 6144 && N <= 512) && (M <= 16 ? K <= 8192 : (int64_t)K * N < 14000000)) return false;
    return stream_plan(M, K, N).slices < 65536;
}

int64_t stream_workspace(int M, int K, int N)
{
    const StreamPlan p = stream_plan(M, K, N);
    return p.slices > 1 ? (int64_t)p.slices * M * N * 4 : 0;
}

template <int BITS, bool PGZ, int RB, bool G128>
static hipError_t stream_launch(const GemvArgs &a, const StreamPlan &p, float *sums, hipStream_t st)
{
    static bool attr_set = false;
    if (!attr_set) {
        hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(&stream_kernel<BITS, PGZ, RB, G128>),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, 160 * 1024);
        if (e != hipSuccess) return e;
        attr_set = true;
    }
    hipLaunchKernelGGL((stream_kernel<BITS, PGZ, RB, G128>), dim3((unsigned)p.groups, (unsigned)p.slices), dim3(64 * p.W),
                       (size_t)p.steps * 4 * 16 * RB * 64, st, a.X, a.wq, a.s, a.z, a.Y, sums, a.M, a.K, a.N, a.G, p.steps, a.ep);
    return hipGetLastError();
}

template <int BITS, bool PGZ, int RB>
static hipError_t stream_groups(const GemvArgs &a, const StreamPlan &p, float *sums, hipStream_t st)
{
    return a.G == 128 ? stream_launch<BITS, PGZ, RB, true>(a, p, sums, st) : stream_launch<BITS, PGZ, RB, false>(a, p, sums, st);
}

template <int BITS, bool PGZ>
static hipError_t stream_go(const GemvArgs &a, float *part, hipStream_t st)
{
    const StreamPlan p = stream_plan(a.M, a.K, a.N);
    float *sums = p.slices > 1 ? part : nullptr;
    hipError_t e = p.RB == 1 ? stream_groups<BITS, PGZ, 1>(a, p, sums, st)
                             : p.RB == 2 ? stream_groups<BITS, PGZ, 2>(a, p, sums, st) : stream_groups<BITS, PGZ, 4>(a, p, sums, st);
    return e != hipSuccess || p.slices == 1 ? e : launch_join(a, part, p.slices, st);
}

hipError_t launch_stream(const GemvArgs &a, float *part, hipStream_t st)
{
    switch (a.bits) {
#define QMM_SB(B) case B: return a.z ? stream_go<B, true>(a, part, st) : stream_go<B, false>(a, part, st);
        QMM_SB(1) QMM_SB(2) QMM_SB(3) QMM_SB(4) QMM_SB(5) QMM_SB(6) QMM_SB(7) QMM_SB(8)
#undef QMM_SB
        default: return hipErrorInvalidValue;
    }
}

}  // namespace qmm
