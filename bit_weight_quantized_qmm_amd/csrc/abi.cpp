// abi.cpp -- the C ABI declared in include/qmm.h: argument validation (host
// only, before any HIP call), then one launch on the caller's stream.
#include "../../include/qmm.h"

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdio.h>
#include <string.h>

#include <initializer_list>
#include <utility>

#include "launch.hpp"

namespace {

thread_local char g_last_error[256] = "";

qmm_status fail(qmm_status st, const char *fmt, const char *what)
{
    snprintf(g_last_error, sizeof g_last_error, fmt, what);
    return st;
}

// Largest sizes the kernels index with 32-bit arithmetic: with K <= 2^21 every
// buffer resource the kernels build (at most 256 rows of X, 64 columns of Wq)
// stays below 2^31 bytes, below the out-of-range offset they use for padding.
constexpr int64_t kMaxK = int64_t(1) << 21;
constexpr int64_t kMaxN = int64_t(1) << 24;
constexpr int64_t kMaxM = int64_t(1) << 24;

qmm_status check_shape(const char *fn, int64_t M, int64_t K, int64_t N, int bits, int64_t G, bool need_g)
{
    if (bits < 1 || bits > 8) return fail(QMM_ERR_INVALID_ARG, "%s: bits must be in 1..8", fn);
    if (K < 32 || K % 32 != 0) return fail(QMM_ERR_INVALID_ARG, "%s: K must be a positive multiple of 32", fn);
    if (N < 1) return fail(QMM_ERR_INVALID_ARG, "%s: N must be >= 1", fn);
    if (M < 1) return fail(QMM_ERR_INVALID_ARG, "%s: M must be >= 1", fn);
    if (need_g && (G < 32 || G % 32 != 0 || K % G != 0))
        return fail(QMM_ERR_INVALID_ARG, "%s: G must be a positive multiple of 32 dividing K", fn);
    if (K > kMaxK || N > kMaxN || M > kMaxM)
        return fail(QMM_ERR_UNSUPPORTED, "%s: dimension beyond the supported range", fn);
    if ((K / 32) * N > (int64_t(1) << 31) - 256)
        return fail(QMM_ERR_UNSUPPORTED, "%s: problem beyond the supported range", fn);
    if (((M + 127) / 128) * ((N + 255) / 256) > (int64_t(1) << 31) - 1)   // GEMM tiles of 128 x 256
        return fail(QMM_ERR_UNSUPPORTED, "%s: problem beyond the supported range", fn);
    return QMM_OK;
}

bool aligned(const void *p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0; }

qmm_status hip_status(hipError_t e, const char *fn)
{
    if (e == hipSuccess) {
        g_last_error[0] = '\0';
        return QMM_OK;
    }
    if (e == hipErrorNotSupported) return fail(QMM_ERR_UNSUPPORTED, "%s: shape not supported by the kernel", fn);
    snprintf(g_last_error, sizeof g_last_error, "%s: %s", fn, hipGetErrorString(e));
    return QMM_ERR_HIP;
}

}  // namespace

extern "C" {

size_t qmm_packed_bytes(int64_t K, int64_t N, int bits)
{
    if (bits < 1 || bits > 8 || K < 0 || N < 0 || (K * bits) % 8 != 0) return 0;
    return (size_t)N * (size_t)K * (size_t)bits / 8u;
}

qmm_status qmm_pack(const uint8_t *codes, uint32_t *wq, int64_t K, int64_t N, int bits, qmm_stream stream)
{
    qmm_status st = check_shape("qmm_pack", 1, K, N, bits, 32, false);
    if (st != QMM_OK) return st;
    if (!codes || !wq) return fail(QMM_ERR_INVALID_ARG, "%s: null pointer", "qmm_pack");
    return hip_status(qmm::launch_pack(codes, wq, (int)K, (int)N, bits, false, (hipStream_t)stream), "qmm_pack");
}

qmm_status qmm_pack_signed(const int8_t *codes, uint32_t *wq, int64_t K, int64_t N, int bits, qmm_stream stream)
{
    const char *fn = "qmm_pack_signed";
    qmm_status st = check_shape(fn, 1, K, N, bits, 32, false);
    if (st != QMM_OK) return st;
    if (!codes || !wq) return fail(QMM_ERR_INVALID_ARG, "%s: null pointer", fn);
    return hip_status(qmm::launch_pack(reinterpret_cast<const uint8_t *>(codes), wq, (int)K, (int)N, bits, true,
                                       (hipStream_t)stream),
                      fn);
}

qmm_status qmm_unpack(const uint32_t *wq, uint8_t *codes, int64_t K, int64_t N, int bits, qmm_stream stream)
{
    qmm_status st = check_shape("qmm_unpack", 1, K, N, bits, 32, false);
    if (st != QMM_OK) return st;
    if (!codes || !wq) return fail(QMM_ERR_INVALID_ARG, "%s: null pointer", "qmm_unpack");
    return hip_status(qmm::launch_unpack(wq, codes, (int)K, (int)N, bits, (hipStream_t)stream), "qmm_unpack");
}

static qmm_status product(const char *fn, bool gemv, const qmm_half *X, const uint32_t *wq, const qmm_half *s,
                          const qmm_half *z, qmm_half *Y, int64_t M, int64_t K, int64_t N, int bits, int64_t G,
                          qmm_stream stream)
{
    qmm_status st = check_shape(fn, M, K, N, bits, G, true);
    if (st != QMM_OK) return st;
    if (gemv && M > 16) return fail(QMM_ERR_INVALID_ARG, "%s: M must be <= 16 (use qmm_gemm)", fn);
    if (!X || !wq || !s || !Y) return fail(QMM_ERR_INVALID_ARG, "%s: null pointer", fn);
    qmm::GemvArgs a{X, wq, s, z, Y, (int)M, (int)K, (int)N, bits, (int)G};
    hipError_t e = gemv ? qmm::launch_gemv(a, (hipStream_t)stream) : qmm::launch_gemm(a, (hipStream_t)stream);
    return hip_status(e, fn);
}

qmm_status qmm_gemv(const qmm_half *X, const uint32_t *wq, const qmm_half *s, const qmm_half *z, qmm_half *Y,
                    int64_t M, int64_t K, int64_t N, int bits, int64_t G, qmm_stream stream)
{
    return product("qmm_gemv", true, X, wq, s, z, Y, M, K, N, bits, G, stream);
}

qmm_status qmm_gemv_grouped(const qmm_gemv_problem *probs, int count, int64_t K, int64_t G, qmm_stream stream)
{
    const char *fn = "qmm_gemv_grouped";
    if (!probs) return fail(QMM_ERR_INVALID_ARG, "%s: null problem array", fn);
    if (count < 1 || count > qmm::QMM_GROUP_MAX) return fail(QMM_ERR_INVALID_ARG, "%s: count must be in 1..16", fn);
    qmm::GroupArgs ga{};
    ga.count = count;
    ga.K = (int)K;
    ga.G = (int)G;
    for (int p = 0; p < count; ++p) {
        const qmm_gemv_problem &q = probs[p];
        qmm_status st = check_shape(fn, 1, K, q.N, q.bits, G, true);
        if (st != QMM_OK) return st;
        if (!q.X || !q.wq || !q.s || !q.Y) return fail(QMM_ERR_INVALID_ARG, "%s: null pointer in a problem", fn);
        if (K > 16384 || (K / 32) * q.N * 4 * (int64_t)q.bits >= (int64_t(1) << 31) - 1)
            return fail(QMM_ERR_UNSUPPORTED, "%s: K <= 16384 and a problem's weights below 2 GiB are supported", fn);
        ga.p[p] = qmm::GroupProblem{q.X, q.wq, q.s, q.z, q.Y, (int)q.N, q.bits};
    }
    return hip_status(qmm::launch_gemv_grouped(ga, (hipStream_t)stream), fn);
}

qmm_status qmm_gemv_lut(const qmm_half *X, const uint32_t *wq, const qmm_half *s, const qmm_half *z, qmm_half *Y,
                        int64_t M, int64_t K, int64_t N, int bits, int64_t G, qmm_stream stream)
{
    const char *fn = "qmm_gemv_lut";
    qmm_status st = check_shape(fn, M, K, N, bits, G, true);
    if (st != QMM_OK) return st;
    if (!X || !wq || !s || !Y) return fail(QMM_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (M != 1 || bits != 1 || K > 8192)
        return fail(QMM_ERR_UNSUPPORTED, "%s: implemented for M = 1, bits = 1, K <= 8192", fn);
    qmm::GemvArgs a{X, wq, s, z, Y, (int)M, (int)K, (int)N, bits, (int)G};
    return hip_status(qmm::launch_gemv_lut(a, (hipStream_t)stream), fn);
}

qmm_status qmm_gemm(const qmm_half *X, const uint32_t *wq, const qmm_half *s, const qmm_half *z, qmm_half *Y,
                    int64_t M, int64_t K, int64_t N, int bits, int64_t G, qmm_stream stream)
{
    return product("qmm_gemm", false, X, wq, s, z, Y, M, K, N, bits, G, stream);
}

qmm_status qmm_gemm_fp(const qmm_half *X, const uint32_t *wq, const qmm_half *s, qmm_half *Y, int64_t M, int64_t K,
                       int64_t N, int fmt, int64_t G, qmm_stream stream)
{
    const char *fn = "qmm_gemm_fp";
    static const int kBits[] = {4, 8, 6, 6, 3, 5, 7};   // by format id (qmm.h)
    if (fmt < QMM_FP4_E2M1 || fmt > QMM_FP7_E3M3) return fail(QMM_ERR_INVALID_ARG, "%s: unknown code format", fn);
    const int bits = kBits[fmt];
    qmm_status st = check_shape(fn, M, K, N, bits, G, true);
    if (st != QMM_OK) return st;
    if (!X || !wq || !s || !Y) return fail(QMM_ERR_INVALID_ARG, "%s: null pointer", fn);
    qmm::GemvArgs a{X, wq, s, nullptr, Y, (int)M, (int)K, (int)N, bits, (int)G};
    const int f = fmt;   // 0 E2M1, 1 E4M3, 2 E3M2, 3 E2M3, 4 E1M1, 5 E2M2, 6 E3M3
    if (M <= 16) {   // the decode kernels where they take the shape
        const hipError_t e = qmm::launch_gemv_fp(a, f, (hipStream_t)stream);
        if (e != hipErrorNotSupported) return hip_status(e, fn);
    }
    return hip_status(qmm::launch_gemm_fp(a, f, (hipStream_t)stream), fn);
}

static qmm_status int8_product(const char *fn, const int8_t *Xq, const qmm_half *sx, const uint32_t *wq,
                               const qmm_half *s, const qmm_half *z, qmm_half *Y, int32_t *acc_out, int64_t M,
                               int64_t K, int64_t N, int bits, int64_t G, qmm_stream stream)
{
    qmm_status st = check_shape(fn, M, K, N, bits, G, true);
    if (st != QMM_OK) return st;
    if (!Xq || !sx || !wq || !s || !Y) return fail(QMM_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (G % 128 != 0 || (G / 128 & (G / 128 - 1)) != 0 || G > 1024)
        return fail(QMM_ERR_UNSUPPORTED, "%s: G must be 128, 256, 512 or 1024", fn);
    if ((M + 15) / 16 > 65535) return fail(QMM_ERR_UNSUPPORTED, "%s: M too large", fn);
    if (acc_out && M * (K / G) * N > (int64_t(1) << 31) - 1)
        return fail(QMM_ERR_UNSUPPORTED, "%s: accumulator dump too large", fn);
    qmm::W4A8Args a{Xq, sx, wq, s, z, Y, acc_out, (int)M, (int)K, (int)N, bits, (int)G};
    return hip_status(qmm::launch_w4a8(a, (hipStream_t)stream), fn);
}

qmm_status qmm_gemm_w4a8(const int8_t *Xq, const qmm_half *sx, const uint32_t *wq, const qmm_half *s,
                         const qmm_half *z, qmm_half *Y, int32_t *acc_out, int64_t M, int64_t K, int64_t N,
                         int64_t G, qmm_stream stream)
{
    return int8_product("qmm_gemm_w4a8", Xq, sx, wq, s, z, Y, acc_out, M, K, N, 4, G, stream);
}

qmm_status qmm_gemm_wka8(const int8_t *Xq, const qmm_half *sx, const uint32_t *wq, const qmm_half *s,
                         const qmm_half *z, qmm_half *Y, int32_t *acc_out, int64_t M, int64_t K, int64_t N, int bits,
                         int64_t G, qmm_stream stream)
{
    return int8_product("qmm_gemm_wka8", Xq, sx, wq, s, z, Y, acc_out, M, K, N, bits, G, stream);
}

qmm_status qmm_quantize(const qmm_half *W, uint8_t *codes, qmm_half *s, qmm_half *z, int64_t K, int64_t N, int bits,
                        int64_t G, qmm_stream stream)
{
    const char *fn = "qmm_quantize";
    qmm_status st = check_shape(fn, 1, K, N, bits, G, true);
    if (st != QMM_OK) return st;
    if (!W || !codes || !s || !z) return fail(QMM_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (K / G > 65535) return fail(QMM_ERR_UNSUPPORTED, "%s: more than 65535 groups per column", fn);
    return hip_status(qmm::launch_quantize(W, codes, s, z, (int)K, (int)N, bits, (int)G, (hipStream_t)stream), fn);
}

static int64_t linear_workspace(int M, int K, int N)
{
    if (qmm::stream_takes(M, K, N)) return qmm::stream_workspace(M, K, N);
    return M <= 16 ? 0 : qmm::gemm_workspace(M, K, N);
}

qmm_status qmm_linear(const qmm_linear_args *p, qmm_stream stream)
{
    const char *fn = "qmm_linear";
    if (!p) return fail(QMM_ERR_INVALID_ARG, "%s: null arguments", fn);
    qmm_status st = check_shape(fn, p->M, p->K, p->N, p->bits, p->G, true);
    if (st != QMM_OK) return st;
    if (!p->X || !p->wq || !p->s || !p->Y) return fail(QMM_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (p->act < QMM_ACT_NONE || p->act > QMM_ACT_GELU_TANH) return fail(QMM_ERR_INVALID_ARG, "%s: unknown activation", fn);
    qmm::GemvArgs a{p->X, p->wq, p->s, p->z, p->Y, (int)p->M, (int)p->K, (int)p->N, p->bits, (int)p->G};
    a.ep = qmm::Epilogue{p->bias, p->mul, p->residual, p->act};
    const int64_t need = linear_workspace(a.M, a.K, a.N);
    if (need > 0 && (!p->workspace || p->workspace_bytes < need || !aligned(p->workspace, 16)))
        return fail(QMM_ERR_INVALID_ARG, "%s: workspace missing, too small or not 16-byte aligned", fn);
    float *part = (float *)p->workspace;
    const hipError_t e = qmm::stream_takes(a.M, a.K, a.N) ? qmm::launch_stream(a, part, (hipStream_t)stream)
                         : a.M <= 16                      ? qmm::launch_gemv_linear(a, (hipStream_t)stream)
                                                          : qmm::launch_gemm_linear(a, part, (hipStream_t)stream);
    return hip_status(e, fn);
}

int64_t qmm_linear_workspace(const qmm_linear_args *p)
{
    if (!p || check_shape("qmm_linear_workspace", p->M, p->K, p->N, p->bits, p->G, true) != QMM_OK) return 0;
    return linear_workspace((int)p->M, (int)p->K, (int)p->N);
}

qmm_status qmm_kv_append(const qmm_kv_append_args *p, qmm_stream stream)
{
    const char *fn = "qmm_kv_append";
    if (!p) return fail(QMM_ERR_INVALID_ARG, "%s: null arguments", fn);
    if (p->T < 0 || p->Hq < 0 || p->Hkv < 1 || p->page < 1 || p->pages < 1)
        return fail(QMM_ERR_INVALID_ARG, "%s: T and Hq must be >= 0, Hkv, page and pages >= 1", fn);
    if (p->D < 2 || p->D % 2 != 0 || p->rot < 0 || p->rot % 2 != 0 || p->rot > p->D)
        return fail(QMM_ERR_INVALID_ARG, "%s: D and rot must be even, 2 <= D, 0 <= rot <= D", fn);
    if (p->dtype != QMM_F16 && p->dtype != QMM_BF16) return fail(QMM_ERR_INVALID_ARG, "%s: dtype must be fp16 or bf16", fn);
    if (p->cache_dtype != p->dtype && p->cache_dtype != QMM_E4M3)
        return fail(QMM_ERR_INVALID_ARG, "%s: the caches must have q's type or e4m3", fn);
    const bool e4m3 = p->cache_dtype == QMM_E4M3;
    const int64_t lim = int64_t(1) << 31;
    if (p->Hq > lim || p->Hkv > lim || p->Hq + 2 * p->Hkv > 65535)
        return fail(QMM_ERR_UNSUPPORTED, "%s: more than 65535 heads", fn);
    if (p->D > 65536 || p->T >= lim || p->T * p->D >= lim || p->page >= lim || p->pages >= lim || p->pages * p->page >= lim)
        return fail(QMM_ERR_UNSUPPORTED, "%s: size beyond the supported range", fn);
    if (p->T == 0) return hip_status(hipSuccess, fn);
    if ((p->Hq > 0 && (!p->q || !p->out)) || !p->k || !p->v || !p->k_cache || !p->v_cache || !p->slots ||
        (p->rot > 0 && (!p->positions || !p->rope)) || (e4m3 && (!p->k_scale || !p->v_scale)))
        return fail(QMM_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (p->rot > 0 && (p->table_rows < 1 || p->table_rows >= lim))
        return fail(QMM_ERR_INVALID_ARG, "%s: the table must have 1 to 2^31 - 1 rows", fn);

    qmm::AppendArgs a{};
    a.q = p->q, a.k = p->k, a.v = p->v, a.out = p->out, a.k_cache = p->k_cache, a.v_cache = p->v_cache;
    a.slots = p->slots, a.positions = p->positions, a.rope = p->rope, a.k_scale = p->k_scale, a.v_scale = p->v_scale;
    a.q_ts = p->q_stride[0], a.q_hs = p->q_stride[1], a.k_ts = p->k_stride[0], a.k_hs = p->k_stride[1];
    a.v_ts = p->v_stride[0], a.v_hs = p->v_stride[1], a.o_ts = p->out_stride[0], a.o_hs = p->out_stride[1];
    a.kc_ps = p->k_cache_stride[0], a.kc_hs = p->k_cache_stride[1], a.kc_ts = p->k_cache_stride[2];
    a.vc_ps = p->v_cache_stride[0], a.vc_hs = p->v_cache_stride[1], a.vc_ts = p->v_cache_stride[2];
    a.T = (int)p->T, a.Hq = (int)p->Hq, a.Hkv = (int)p->Hkv, a.D = (int)p->D, a.rot = (int)p->rot;
    a.page = (int)p->page, a.pages = (int)p->pages, a.table_rows = (int)p->table_rows, a.pairs = p->pairs != 0;

    // widest vector at whose multiples every row and every half of the pairs stands
    auto fits = [&](int64_t v) {
        if (p->rot % (2 * v) != 0 || (p->D - p->rot) % (2 * v) != 0) return false;
        for (const int64_t *sd : {p->k_stride, p->v_stride, p->q_stride, p->out_stride})
            if ((p->Hq > 0 || sd == p->k_stride || sd == p->v_stride) && (sd[0] % v != 0 || sd[1] % v != 0)) return false;
        for (const int64_t *sd : {p->k_cache_stride, p->v_cache_stride})
            if (sd[0] % v != 0 || sd[1] % v != 0 || sd[2] % v != 0) return false;
        if (p->Hq > 0 && (!aligned(p->q, 2 * v) || !aligned(p->out, 2 * v))) return false;
        const int64_t cell = e4m3 ? 1 : 2;
        return aligned(p->k, 2 * v) && aligned(p->v, 2 * v) && aligned(p->k_cache, cell * v) && aligned(p->v_cache, cell * v) &&
               aligned(p->rope, 16);
    };
    const int vec = fits(8) ? 8 : fits(4) ? 4 : 1;
    return hip_status(qmm::launch_append(a, p->dtype == QMM_BF16, e4m3, vec, (hipStream_t)stream), fn);
}

// Sizes and types of an attention call; fills what the planner reads.
static qmm_status attention_shape(const char *fn, const qmm_attention_args *p, qmm::AttendArgs &a)
{
    if (!p) return fail(QMM_ERR_INVALID_ARG, "%s: null arguments", fn);
    if (p->T < 0 || p->B < 0 || p->Hq < 1 || p->Hkv < 1 || p->page < 1 || p->pages < 1 || p->width < 1 || p->D < 1)
        return fail(QMM_ERR_INVALID_ARG, "%s: T and B must be >= 0, the other sizes >= 1", fn);
    if (p->max_q < 1 || p->max_kv < 0) return fail(QMM_ERR_INVALID_ARG, "%s: max_q must be >= 1, max_kv >= 0", fn);
    if (p->Hq % p->Hkv != 0) return fail(QMM_ERR_INVALID_ARG, "%s: Hq must be a multiple of Hkv", fn);
    if (p->window < 0) return fail(QMM_ERR_INVALID_ARG, "%s: window must be >= 0", fn);
    if (!(p->scale >= 0) || !isfinite((float)p->scale)) return fail(QMM_ERR_INVALID_ARG, "%s: scale must be finite and >= 0", fn);
    if (p->dtype != QMM_F16 && p->dtype != QMM_BF16) return fail(QMM_ERR_INVALID_ARG, "%s: dtype must be fp16 or bf16", fn);
    if (p->cache_dtype != p->dtype && p->cache_dtype != QMM_E4M3)
        return fail(QMM_ERR_INVALID_ARG, "%s: the caches must have q's type or e4m3", fn);
    if (p->D % 16 != 0 || p->D > 256) return fail(QMM_ERR_UNSUPPORTED, "%s: D must be a multiple of 16 up to 256", fn);
    const int64_t lim = (int64_t(1) << 31) - 65536;
    if (p->T > lim || p->B > lim || p->Hq > 65536 || p->page > (1 << 20) || p->pages > lim || p->width > lim ||
        p->max_q > lim || p->max_kv > lim)
        return fail(QMM_ERR_UNSUPPORTED, "%s: size beyond the supported range", fn);
    a.T = (int)p->T, a.B = (int)p->B, a.Hq = (int)p->Hq, a.Hkv = (int)p->Hkv, a.g = (int)(p->Hq / p->Hkv), a.D = (int)p->D;
    a.page = (int)p->page, a.pages = (int)p->pages, a.width = (int)p->width;
    // no sequence has more new tokens than there are rows: smaller bounds, smaller grids
    a.max_q = (int)(p->T > 0 && p->T < p->max_q ? p->T : p->max_q);
    a.max_kv = (int)p->max_kv;
    a.window = (int)(p->window > lim ? 0 : p->window);
    a.scale = (float)p->scale;
    if (p->T * p->Hq > lim || (int64_t)a.max_q * p->Hq > lim) return fail(QMM_ERR_UNSUPPORTED, "%s: size beyond the supported range", fn);
    return QMM_OK;
}

int64_t qmm_paged_attention_workspace(const qmm_attention_args *args)
{
    qmm::AttendArgs a{};
    if (attention_shape("qmm_paged_attention_workspace", args, a) != QMM_OK || a.T == 0 || a.B == 0) return 0;
    return qmm::plan_attend(a, args->cache_dtype == QMM_E4M3);
}

qmm_status qmm_paged_attention(const qmm_attention_args *p, qmm_stream stream)
{
    const char *fn = "qmm_paged_attention";
    qmm::AttendArgs a{};
    qmm_status st = attention_shape(fn, p, a);
    if (st != QMM_OK) return st;
    if (a.T == 0 || a.B == 0) return hip_status(hipSuccess, fn);
    const bool e4m3 = p->cache_dtype == QMM_E4M3;
    if (!p->q || !p->k_cache || !p->v_cache || !p->out || !p->page_table || !p->cu_q || !p->kv_lens ||
        (e4m3 && (!p->k_scale || !p->v_scale)))
        return fail(QMM_ERR_INVALID_ARG, "%s: null pointer", fn);
    const int64_t cell = e4m3 ? 1 : 2;
    bool even = aligned(p->q, 16) && aligned(p->k_cache, 16) && aligned(p->v_cache, 16) && aligned(p->out, 16);
    for (int i = 0; i < 2; ++i) even = even && p->q_stride[i] * 2 % 16 == 0 && p->out_stride[i] * 2 % 16 == 0;
    for (int i = 0; i < 3; ++i) even = even && p->k_cache_stride[i] * cell % 16 == 0 && p->v_cache_stride[i] * cell % 16 == 0;
    if (!even) return fail(QMM_ERR_INVALID_ARG, "%s: starts and strides must be multiples of 16 bytes", fn);
    const int64_t kt = p->k_cache_stride[2] * cell, vt = p->v_cache_stride[2] * cell;
    if (kt < 0 || vt < 0 || kt > (1 << 24) || vt > (1 << 24))   // 64 tokens of it stay below 2^31
        return fail(QMM_ERR_UNSUPPORTED, "%s: token strides of the caches must be 0 to 2^24 bytes", fn);
    a.q = p->q, a.k = p->k_cache, a.v = p->v_cache, a.out = p->out, a.lse = p->lse;
    a.table = p->page_table, a.cu_q = p->cu_q, a.kv_lens = p->kv_lens, a.k_scale = p->k_scale, a.v_scale = p->v_scale;
    a.q_ts = p->q_stride[0] * 2, a.q_hs = p->q_stride[1] * 2, a.o_ts = p->out_stride[0] * 2, a.o_hs = p->out_stride[1] * 2;
    a.k_ps = p->k_cache_stride[0] * cell, a.k_hs = p->k_cache_stride[1] * cell, a.k_ts = (uint32_t)kt;
    a.v_ps = p->v_cache_stride[0] * cell, a.v_hs = p->v_cache_stride[1] * cell, a.v_ts = (uint32_t)vt;
    a.table_s = p->table_stride;
    const int64_t need = qmm::plan_attend(a, e4m3);
    if (need > 0 && (!p->workspace || p->workspace_bytes < need || !aligned(p->workspace, 16)))
        return fail(QMM_ERR_INVALID_ARG, "%s: workspace missing, too small or not 16-byte aligned", fn);
    a.part = (float *)p->workspace;
    return hip_status(qmm::launch_attend(a, p->dtype == QMM_BF16, e4m3, (hipStream_t)stream), fn);
}

// A cache of 4-bit codes: sizes, groups, then pointers and strides.
static qmm_status kv4_shape(const char *fn, const qmm_kv4_cache &c)
{
    if (c.Hkv < 1 || c.page < 1 || c.pages < 1 || c.D < 1 || c.G < 1)
        return fail(QMM_ERR_INVALID_ARG, "%s: the cache's sizes must be >= 1", fn);
    if (c.D % c.G != 0) return fail(QMM_ERR_INVALID_ARG, "%s: D must be a multiple of G", fn);
    if ((c.G != 32 && c.G != 64 && c.G != 128) || c.D > 256)
        return fail(QMM_ERR_UNSUPPORTED, "%s: G must be 32, 64 or 128, D a multiple of it up to 256", fn);
    const int64_t lim = int64_t(1) << 31;
    if (c.Hkv > 65535 || c.page > (1 << 20) || c.pages >= lim || c.pages * c.page >= lim)
        return fail(QMM_ERR_UNSUPPORTED, "%s: size beyond the supported range", fn);
    return QMM_OK;
}
static qmm_status kv4_places(const char *fn, const qmm_kv4_cache &c)
{
    if (!c.k || !c.v || !c.k_scale || !c.v_scale) return fail(QMM_ERR_INVALID_ARG, "%s: null pointer", fn);
    bool even = aligned(c.k, 16) && aligned(c.v, 16) && aligned(c.k_scale, 4) && aligned(c.v_scale, 4);
    for (int i = 0; i < 3; ++i) even = even && c.k_stride[i] % 16 == 0 && c.v_stride[i] % 16 == 0;
    for (int i = 0; i < 2; ++i) even = even && c.k_scale_stride[i] % 2 == 0 && c.v_scale_stride[i] % 2 == 0;
    if (!even)
        return fail(QMM_ERR_INVALID_ARG, "%s: codes must start at multiples of 16 bytes, scales at multiples of 4", fn);
    if (c.k_stride[2] < 0 || c.v_stride[2] < 0 || c.k_stride[2] > (1 << 24) || c.v_stride[2] > (1 << 24))   // 64 tokens of it stay below 2^31
        return fail(QMM_ERR_UNSUPPORTED, "%s: token strides of the codes must be 0 to 2^24 bytes", fn);
    return QMM_OK;
}
static qmm_status heads_shape(const char *fn, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t rot, int64_t table_rows, double eps, int dtype)
{
    if (T < 0 || Hq < 0 || Hkv < 0) return fail(QMM_ERR_INVALID_ARG, "%s: T and the heads must be >= 0", fn);
    if (D < 1 || rot < 0 || rot % 2 != 0 || rot > D) return fail(QMM_ERR_INVALID_ARG, "%s: D >= 1, rot even and 0 to D", fn);
    if (!(eps >= 0) || !isfinite((float)eps)) return fail(QMM_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", fn);
    if (dtype != QMM_F16 && dtype != QMM_BF16) return fail(QMM_ERR_INVALID_ARG, "%s: dtype must be fp16 or bf16", fn);
    if (D % 16 != 0 || rot % 16 != 0 || D > 256) return fail(QMM_ERR_UNSUPPORTED, "%s: D and rot must be multiples of 16, D up to 256", fn);
    const int64_t lim = int64_t(1) << 31;
    if (Hq > 65535 || Hkv > 65535 || Hq + 2 * Hkv > 65535) return fail(QMM_ERR_UNSUPPORTED, "%s: more than 65535 heads", fn);
    if (T >= lim) return fail(QMM_ERR_UNSUPPORTED, "%s: size beyond the supported range", fn);
    if (rot > 0 && (table_rows < 1 || table_rows >= lim)) return fail(QMM_ERR_INVALID_ARG, "%s: the table must have 1 to 2^31 - 1 rows", fn);
    return QMM_OK;
}
// whether the rows of tensors [tokens][heads][D] stand at multiples of 16 bytes
static bool even_rows(std::initializer_list<std::pair<const void *, const int64_t *>> tensors)
{
    for (const auto &t : tensors)
        if (t.first && (!aligned(t.first, 16) || t.second[0] % 8 != 0 || t.second[1] % 8 != 0)) return false;
    return true;
}

qmm_status qmm_qk_norm(const qmm_qk_norm_args *p, qmm_stream stream)
{
    const char *fn = "qmm_qk_norm";
    if (!p) return fail(QMM_ERR_INVALID_ARG, "%s: null arguments", fn);
    qmm_status st = heads_shape(fn, p->T, p->Hq, p->Hkv, p->D, p->rot, p->table_rows, p->eps, p->dtype);
    if (st != QMM_OK) return st;
    if (p->T == 0 || p->Hq + p->Hkv == 0) return hip_status(hipSuccess, fn);
    if ((p->Hq > 0 && (!p->q || !p->q_out)) || (p->Hkv > 0 && (!p->k || !p->k_out)) || (p->rot > 0 && (!p->positions || !p->rope)))
        return fail(QMM_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(p->q_weight, 16) || !aligned(p->k_weight, 16) || !aligned(p->rope, 16))
        return fail(QMM_ERR_INVALID_ARG, "%s: weights and table must start at multiples of 16 bytes", fn);
    qmm::HeadsArgs a{};
    a.q = p->q, a.k = p->k, a.q_out = p->q_out, a.k_out = p->k_out, a.q_weight = p->q_weight, a.k_weight = p->k_weight;
    a.positions = p->positions, a.rope = p->rope;
    a.q_ts = p->q_stride[0], a.q_hs = p->q_stride[1], a.k_ts = p->k_stride[0], a.k_hs = p->k_stride[1];
    a.qo_ts = p->q_out_stride[0], a.qo_hs = p->q_out_stride[1], a.ko_ts = p->k_out_stride[0], a.ko_hs = p->k_out_stride[1];
    a.T = (int)p->T, a.Hq = (int)p->Hq, a.Hk = (int)p->Hkv, a.D = (int)p->D, a.rot = (int)p->rot, a.table_rows = (int)p->table_rows;
    a.eps = p->eps, a.pairs = p->pairs != 0;
    const bool vec = even_rows({{p->Hq ? p->q : nullptr, p->q_stride}, {p->Hkv ? p->k : nullptr, p->k_stride}, {p->Hq ? p->q_out : nullptr, p->q_out_stride},
                                {p->Hkv ? p->k_out : nullptr, p->k_out_stride}});
    return hip_status(qmm::launch_heads(a, p->dtype == QMM_BF16, vec, false, (hipStream_t)stream), fn);
}

qmm_status qmm_kv4_append(const qmm_kv4_append_args *p, qmm_stream stream)
{
    const char *fn = "qmm_kv4_append";
    if (!p) return fail(QMM_ERR_INVALID_ARG, "%s: null arguments", fn);
    const qmm_kv4_cache &c = p->cache;
    qmm_status st = kv4_shape(fn, c);
    if (st == QMM_OK) st = heads_shape(fn, p->T, p->Hq, c.Hkv, c.D, p->rot, p->table_rows, p->eps, p->dtype);
    if (st != QMM_OK) return st;
    if (p->T == 0) return hip_status(hipSuccess, fn);
    if ((p->Hq > 0 && (!p->q || !p->out)) || !p->k || !p->v || !p->slots || (p->rot > 0 && (!p->positions || !p->rope)))
        return fail(QMM_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (!aligned(p->q_norm, 16) || !aligned(p->k_norm, 16) || !aligned(p->rope, 16))
        return fail(QMM_ERR_INVALID_ARG, "%s: weights and table must start at multiples of 16 bytes", fn);
    if ((st = kv4_places(fn, c)) != QMM_OK) return st;
    qmm::HeadsArgs a{};
    a.q = p->q, a.k = p->k, a.v = p->v, a.q_out = p->out, a.q_weight = p->q_norm, a.k_weight = p->k_norm;
    a.positions = p->positions, a.rope = p->rope, a.slots = p->slots;
    a.k_codes = c.k, a.v_codes = c.v, a.k_scale = c.k_scale, a.v_scale = c.v_scale;
    a.q_ts = p->q_stride[0], a.q_hs = p->q_stride[1], a.k_ts = p->k_stride[0], a.k_hs = p->k_stride[1];
    a.v_ts = p->v_stride[0], a.v_hs = p->v_stride[1], a.qo_ts = p->out_stride[0], a.qo_hs = p->out_stride[1];
    a.kc_ps = c.k_stride[0], a.kc_hs = c.k_stride[1], a.kc_ts = c.k_stride[2], a.vc_ps = c.v_stride[0], a.vc_hs = c.v_stride[1], a.vc_ts = c.v_stride[2];
    a.ks_ps = c.k_scale_stride[0], a.ks_hs = c.k_scale_stride[1], a.vs_ps = c.v_scale_stride[0], a.vs_hs = c.v_scale_stride[1];
    a.T = (int)p->T, a.Hq = (int)p->Hq, a.Hk = 0, a.Hkv = (int)c.Hkv, a.D = (int)c.D, a.G = (int)c.G, a.rot = (int)p->rot;
    a.page = (int)c.page, a.pages = (int)c.pages, a.table_rows = (int)p->table_rows, a.eps = p->eps, a.pairs = p->pairs != 0;
    const bool vec = even_rows({{p->k, p->k_stride}, {p->v, p->v_stride}, {p->Hq ? p->q : nullptr, p->q_stride}, {p->Hq ? p->out : nullptr, p->out_stride}});
    return hip_status(qmm::launch_heads(a, p->dtype == QMM_BF16, vec, true, (hipStream_t)stream), fn);
}

qmm_status qmm_kv4_read(const qmm_kv4_read_args *p, qmm_stream stream)
{
    const char *fn = "qmm_kv4_read";
    if (!p) return fail(QMM_ERR_INVALID_ARG, "%s: null arguments", fn);
    const qmm_kv4_cache &c = p->cache;
    qmm_status st = kv4_shape(fn, c);
    if (st != QMM_OK) return st;
    if (p->T < 0) return fail(QMM_ERR_INVALID_ARG, "%s: T must be >= 0", fn);
    if (p->dtype != QMM_F16 && p->dtype != QMM_BF16) return fail(QMM_ERR_INVALID_ARG, "%s: dtype must be fp16 or bf16", fn);
    if (p->T >= (int64_t(1) << 31)) return fail(QMM_ERR_UNSUPPORTED, "%s: size beyond the supported range", fn);
    if (p->T == 0) return hip_status(hipSuccess, fn);
    if (!p->slots || !p->k_out || !p->v_out) return fail(QMM_ERR_INVALID_ARG, "%s: null pointer", fn);
    if ((st = kv4_places(fn, c)) != QMM_OK) return st;
    qmm::Read4Args a{};
    a.k_codes = c.k, a.v_codes = c.v, a.k_scale = c.k_scale, a.v_scale = c.v_scale, a.slots = p->slots, a.k_out = p->k_out, a.v_out = p->v_out;
    a.kc_ps = c.k_stride[0], a.kc_hs = c.k_stride[1], a.kc_ts = c.k_stride[2], a.vc_ps = c.v_stride[0], a.vc_hs = c.v_stride[1], a.vc_ts = c.v_stride[2];
    a.ks_ps = c.k_scale_stride[0], a.ks_hs = c.k_scale_stride[1], a.vs_ps = c.v_scale_stride[0], a.vs_hs = c.v_scale_stride[1];
    a.ko_ts = p->k_out_stride[0], a.ko_hs = p->k_out_stride[1], a.vo_ts = p->v_out_stride[0], a.vo_hs = p->v_out_stride[1];
    a.T = (int)p->T, a.Hkv = (int)c.Hkv, a.D = (int)c.D, a.lg_G = c.G == 32 ? 5 : c.G == 64 ? 6 : 7, a.page = (int)c.page, a.pages = (int)c.pages;
    a.by_page.set(c.page);
    return hip_status(qmm::launch_read4(a, p->dtype == QMM_BF16, even_rows({{p->k_out, p->k_out_stride}, {p->v_out, p->v_out_stride}}), (hipStream_t)stream), fn);
}

// Sizes and types of an attention call over 4-bit codes; fills what the planner reads.
static qmm_status attention4_shape(const char *fn, const qmm_kv4_attention_args *p, qmm::Attend4Args &a)
{
    if (!p) return fail(QMM_ERR_INVALID_ARG, "%s: null arguments", fn);
    const qmm_kv4_cache &c = p->cache;
    qmm_status st = kv4_shape(fn, c);
    if (st != QMM_OK) return st;
    if (p->T < 0 || p->B < 0 || p->Hq < 1 || p->width < 1)
        return fail(QMM_ERR_INVALID_ARG, "%s: T and B must be >= 0, the other sizes >= 1", fn);
    if (p->max_q < 1 || p->max_kv < 0) return fail(QMM_ERR_INVALID_ARG, "%s: max_q must be >= 1, max_kv >= 0", fn);
    if (p->Hq % c.Hkv != 0) return fail(QMM_ERR_INVALID_ARG, "%s: Hq must be a multiple of Hkv", fn);
    if (p->window < 0 || p->sinks < 0) return fail(QMM_ERR_INVALID_ARG, "%s: window and sinks must be >= 0", fn);
    if (!(p->scale >= 0) || !isfinite((float)p->scale)) return fail(QMM_ERR_INVALID_ARG, "%s: scale must be finite and >= 0", fn);
    if (p->dtype != QMM_F16 && p->dtype != QMM_BF16) return fail(QMM_ERR_INVALID_ARG, "%s: dtype must be fp16 or bf16", fn);
    const int64_t lim = (int64_t(1) << 31) - 65536;
    if (p->T > lim || p->B > lim || p->Hq > 65536 || p->width > lim || p->max_q > lim || p->max_kv > lim)
        return fail(QMM_ERR_UNSUPPORTED, "%s: size beyond the supported range", fn);
    a.T = (int)p->T, a.B = (int)p->B, a.Hq = (int)p->Hq, a.Hkv = (int)c.Hkv, a.g = (int)(p->Hq / c.Hkv), a.D = (int)c.D;
    a.lg_G = c.G == 32 ? 5 : c.G == 64 ? 6 : 7, a.s_ts = (uint32_t)(4 * (c.D / c.G));
    a.page = (int)c.page, a.pages = (int)c.pages, a.width = (int)p->width;
    // no sequence has more new tokens than there are rows: smaller bounds, smaller grids
    a.max_q = (int)(p->T > 0 && p->T < p->max_q ? p->T : p->max_q);
    a.max_kv = (int)p->max_kv;
    a.window = (int)(p->window > lim ? 0 : p->window);
    a.sinks = a.window > 0 ? (int)(p->sinks > lim ? lim : p->sinks) : 0;   // without a window every key before a row is seen
    a.scale = (float)p->scale;
    a.halves = c.page % 16 == 0;
    if (p->T * p->Hq > lim || (int64_t)a.max_q * p->Hq > lim) return fail(QMM_ERR_UNSUPPORTED, "%s: size beyond the supported range", fn);
    return QMM_OK;
}

int64_t qmm_kv4_attention_workspace(const qmm_kv4_attention_args *args)
{
    qmm::Attend4Args a{};
    if (attention4_shape("qmm_kv4_attention_workspace", args, a) != QMM_OK || a.T == 0 || a.B == 0) return 0;
    return qmm::plan_attend4(a);
}

qmm_status qmm_kv4_attention(const qmm_kv4_attention_args *p, qmm_stream stream)
{
    const char *fn = "qmm_kv4_attention";
    qmm::Attend4Args a{};
    qmm_status st = attention4_shape(fn, p, a);
    if (st != QMM_OK) return st;
    if (a.T == 0 || a.B == 0) return hip_status(hipSuccess, fn);
    const qmm_kv4_cache &c = p->cache;
    if (!p->q || !p->out || !p->page_table || !p->cu_q || !p->kv_lens) return fail(QMM_ERR_INVALID_ARG, "%s: null pointer", fn);
    bool even = aligned(p->q, 16) && aligned(p->out, 16);
    for (int i = 0; i < 2; ++i) even = even && p->q_stride[i] % 8 == 0 && p->out_stride[i] % 8 == 0;
    if (!even) return fail(QMM_ERR_INVALID_ARG, "%s: starts and strides of q and out must be multiples of 16 bytes", fn);
    if ((st = kv4_places(fn, c)) != QMM_OK) return st;
    a.q = p->q, a.k = c.k, a.v = c.v, a.ks = c.k_scale, a.vs = c.v_scale, a.out = p->out, a.lse = p->lse;
    a.table = p->page_table, a.cu_q = p->cu_q, a.kv_lens = p->kv_lens;
    a.q_ts = p->q_stride[0] * 2, a.q_hs = p->q_stride[1] * 2, a.o_ts = p->out_stride[0] * 2, a.o_hs = p->out_stride[1] * 2;
    a.k_ps = c.k_stride[0], a.k_hs = c.k_stride[1], a.k_ts = (uint32_t)c.k_stride[2];
    a.v_ps = c.v_stride[0], a.v_hs = c.v_stride[1], a.v_ts = (uint32_t)c.v_stride[2];
    a.ks_ps = c.k_scale_stride[0] * 2, a.ks_hs = c.k_scale_stride[1] * 2, a.vs_ps = c.v_scale_stride[0] * 2, a.vs_hs = c.v_scale_stride[1] * 2;
    a.table_s = p->table_stride;
    const int64_t need = qmm::plan_attend4(a);
    if (need > 0 && (!p->workspace || p->workspace_bytes < need || !aligned(p->workspace, 16)))
        return fail(QMM_ERR_INVALID_ARG, "%s: workspace missing, too small or not 16-byte aligned", fn);
    a.part = (float *)p->workspace;
    return hip_status(qmm::launch_attend4(a, p->dtype == QMM_BF16, (hipStream_t)stream), fn);
}

qmm_status qmm_probe_read(const void *buf, uint64_t bytes, uint32_t *sink, int grid, qmm_stream stream)
{
    const char *fn = "qmm_probe_read";
    if (!buf || !sink) return fail(QMM_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (bytes < 16 || bytes % 16 != 0) return fail(QMM_ERR_INVALID_ARG, "%s: bytes must be a positive multiple of 16", fn);
    if (grid < 1 || grid > 65535) return fail(QMM_ERR_INVALID_ARG, "%s: grid must be in 1..65535", fn);
    return hip_status(qmm::launch_probe_read(buf, bytes, sink, grid, (hipStream_t)stream), fn);
}

qmm_status qmm_probe_mfma(float *sink, int iters, int grid, int shape, qmm_stream stream)
{
    const char *fn = "qmm_probe_mfma";
    if (!sink) return fail(QMM_ERR_INVALID_ARG, "%s: null pointer", fn);
    if (iters < 1 || grid < 1 || grid > 65535 || (shape != 0 && shape != 1))
        return fail(QMM_ERR_INVALID_ARG, "%s: iters >= 1, grid in 1..65535, shape 0 or 1", fn);
    return hip_status(qmm::launch_probe_mfma(sink, iters, grid, shape, (hipStream_t)stream), fn);
}

const char *qmm_status_string(qmm_status status)
{
    switch (status) {
        case QMM_OK: return "ok";
        case QMM_ERR_INVALID_ARG: return "invalid argument";
        case QMM_ERR_UNSUPPORTED: return "unsupported shape";
        case QMM_ERR_HIP: return "HIP launch failure";
        default: return "unknown status";
    }
}

const char *qmm_last_error(void) { return g_last_error; }

const char *qmm_last_hip_error(void) { return g_last_error; }

}  // extern "C"
