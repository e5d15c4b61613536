// launch.hpp -- internal launchers behind the C ABI (arguments already validated).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmm {

// Y = act(product + bias) * mul + residual (qmm_linear); null: not there
enum { ACT_NONE = 0, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH };
struct Epilogue {
    const uint16_t *bias;      // fp16 [N]
    const uint16_t *mul;       // fp16 [M][N]
    const uint16_t *residual;  // fp16 [M][N]
    int act;
};

struct GemvArgs {
    const uint16_t *X;     // fp16 [M][K]
    const uint32_t *wq;    // [N][K*bits/32]
    const uint16_t *s;     // fp16 [N][K/G]
    const uint16_t *z;     // fp16 [N][K/G] or nullptr
    uint16_t *Y;           // fp16 [M][N]
    int M, K, N, bits, G;
    Epilogue ep = {};      // qmm_linear's launchers alone read it
};

struct W4A8Args {
    const int8_t *Xq;      // [M][K]
    const uint16_t *sx;    // fp16 [M]
    const uint32_t *wq;    // [N][K*bits/32]
    const uint16_t *s;     // fp16 [N][K/G]
    const uint16_t *z;     // fp16 [N][K/G] or nullptr
    uint16_t *Y;           // fp16 [M][N]
    int32_t *acc;          // int32 [M][K/G][N] or nullptr
    int M, K, N, bits, G;
};

// Grouped M = 1 products (qmm_gemv_grouped): one launch, every problem with
// the same K and G, its own X, weights, scales, zero-points, output, N and
// code width.
constexpr int QMM_GROUP_MAX = 16;
struct GroupProblem {
    const uint16_t *X;     // fp16 [1][K]
    const uint32_t *wq;    // [N][K*bits/32]
    const uint16_t *s;     // fp16 [N][K/G]
    const uint16_t *z;     // fp16 [N][K/G] or nullptr
    uint16_t *Y;           // fp16 [1][N]
    int N, bits;
};
struct GroupArgs {
    GroupProblem p[QMM_GROUP_MAX];
    int wg0[QMM_GROUP_MAX + 1];   // workgroups of problem p: wg0[p] .. wg0[p + 1] - 1 (set by the launcher)
    int count, K, G;
};

// Rotary positions and the append to a paged cache (qmm_kv_append).  Strides in elements.
struct AppendArgs {
    const void *q, *k, *v;
    void *out, *k_cache, *v_cache;
    const int64_t *slots;
    const int32_t *positions;
    const float *rope, *k_scale, *v_scale;
    int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs;
    int64_t kc_ps, kc_hs, kc_ts, vc_ps, vc_hs, vc_ts;
    int T, Hq, Hkv, D, rot, page, pages, table_rows;
    bool pairs;
};

// Attention over a paged cache (qmm_paged_attention).  Strides in bytes.
struct AttendArgs {
    const void *q, *k, *v;
    void *out;
    float *lse;             // [T][Hq] or nullptr
    const int32_t *table, *cu_q, *kv_lens;
    const float *k_scale, *v_scale;
    float *part;            // splits > 1: outputs [T * Hq][splits][D], then log sums [T * Hq][splits]
    int64_t q_ts, q_hs, o_ts, o_hs, k_ps, k_hs, v_ps, v_hs, table_s;
    uint32_t k_ts, v_ts;
    int B, T, Hq, Hkv, g, D, page, width, pages, max_q, max_kv, window;
    uint32_t page_mul;      // key / page = key * page_mul >> page_sh (set by the planner)
    int page_sh;
    int rows;               // query rows (token, head of the group) a workgroup takes
    int rblocks, splits, chunk;
    float scale;
};

hipError_t launch_append(const AppendArgs &a, bool bf16, bool e4m3, int vec, hipStream_t st);
// Chooses the kernel's shape from the sizes (no GPU call): fills rows, rblocks, splits and chunk.
// Returns the bytes of workspace that the launch needs.
int64_t plan_attend(AttendArgs &a, bool e4m3);
hipError_t launch_attend(const AttendArgs &a, bool bf16, bool e4m3, hipStream_t st);

hipError_t launch_pack(const uint8_t *codes, uint32_t *wq, int K, int N, int bits, bool is_signed, hipStream_t st);
hipError_t launch_unpack(const uint32_t *wq, uint8_t *codes, int K, int N, int bits, hipStream_t st);
hipError_t launch_gemv(const GemvArgs &a, hipStream_t st);
hipError_t launch_gemm(const GemvArgs &a, hipStream_t st);
hipError_t launch_gemv_linear(const GemvArgs &a, hipStream_t st);   // with a.ep; M <= 16
hipError_t launch_gemm_linear(const GemvArgs &a, float *part, hipStream_t st);   // with a.ep; part: gemm_workspace() bytes
int64_t gemm_workspace(int M, int K, int N);
// qmm_linear for 2 <= M <= 64 (part: stream_workspace() bytes of fp32 sums)
bool stream_takes(int M, int K, int N);
int64_t stream_workspace(int M, int K, int N);
hipError_t launch_stream(const GemvArgs &a, float *part, hipStream_t st);
hipError_t launch_join(const GemvArgs &a, const float *part, int slices, hipStream_t st);   // slices' sums, epilogue
hipError_t launch_gemm_fp(const GemvArgs &a, int fmt, hipStream_t st);
hipError_t launch_gemv_grouped(const GroupArgs &a, hipStream_t st);
hipError_t launch_gemv_lut(const GemvArgs &a, hipStream_t st);   // M = 1, 1-bit codes; NotSupported otherwise
hipError_t launch_gemv_fp(const GemvArgs &a, int fmt, hipStream_t st);   // M <= 16; NotSupported otherwise
hipError_t launch_w4a8(const W4A8Args &a, hipStream_t st);
hipError_t launch_probe_read(const void *buf, uint64_t bytes, uint32_t *sink, int grid, hipStream_t st);
hipError_t launch_probe_mfma(float *sink, int iters, int grid, int shape, hipStream_t st);
hipError_t launch_quantize(const uint16_t *W, uint8_t *codes, uint16_t *s, uint16_t *z, int K, int N, int bits, int G,
                           hipStream_t st);

}  // namespace qmm
