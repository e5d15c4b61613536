// epilogue.hpp -- what follows a product in the same kernel:
//
//     Y = act(h + bias) * mul + residual,   h the product's fp32 sum,
//
// all of it in fp32, rounded once to fp16 at the store.  The file is included
// by the product kernels' sources, which are compiled twice: without
// QMM_EPILOGUE for the plain products, whose code it leaves as it is, and with
// it for qmm_linear.  7B gate projection (1 x 4096 x 11008, 4 bits, silu, mul): 5.9 us a
// call; prompt of 4096 rows (4096 x 14336): 545 us, 883 TFLOP/s, the operands of the
// epilogue read and Y written 16 bytes a lane from sums that go through LDS.
#pragma once

#include "launch.hpp"
#include "qmm_device.hpp"

#ifdef QMM_EPILOGUE
#define QMM_EPI_PARAM , const Epilogue ep
#define QMM_EPI_ARG , a.ep
#else
#define QMM_EPI_PARAM
#define QMM_EPI_ARG
#endif

namespace qmm {

// Standard normal distribution at -|x|, by erfc: Phi(-|x|) = erfc(t) / 2, t = |x| / sqrt 2,
// erfc(t) = exp(-t^2) erfcx(t), erfcx(t) = u P(u) with u = 1 / (1 + 0.38 t) and P of
// degree 6, fitted here to the smallest largest relative error over 0 <= t <= 14 (1.0e-6; Phi
// has left fp32 there).  Relative accuracy in the tail matters: gelu(x) = x Phi(x) keeps it.
__device__ __forceinline__ float normal_tail(float x)
{
    const float t = __builtin_fabsf(x) * 0.70710678f;
    const float u = __builtin_amdgcn_rcpf(fmaf(0.38f, t, 1.f));
    float p = -0.12541856f;
    p = fmaf(p, u, 0.336039966f);
    p = fmaf(p, u, -0.0699185991f);
    p = fmaf(p, u, 0.247838405f);
    p = fmaf(p, u, 0.180592747f);
    p = fmaf(p, u, 0.216577716f);
    p = fmaf(p, u, 0.21428729f);
    return 0.5f * __builtin_amdgcn_exp2f(-1.44269504f * t * t) * (p * u);
}

// act is uniform over the launch: the compiler's branches on it are scalar
__device__ __forceinline__ float activate(float h, int act)
{
    switch (act) {
        case ACT_RELU: return h < 0.f ? 0.f : h;   // NaN passes
        case ACT_SILU: return h * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.44269504f * h));
        case ACT_GELU: {
            const float q = normal_tail(h);
            return h * (h < 0.f ? q : 1.f - q);
        }
        case ACT_GELU_TANH: {   // (1 + tanh y) / 2 = 1 / (1 + exp(-2y))
            const float y = 0.79788456f * fmaf(0.044715f * h * h, h, h);
            return h * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-2.88539008f * y));
        }
        default: return h;
    }
}

// 8 fp16 at any element: rows of an odd number of columns start at 2-byte
// multiples, where the 16-byte accesses still work, across two lines at times
typedef _Float16 half8u_t __attribute__((ext_vector_type(8), aligned(2)));
__device__ __forceinline__ half8_t load_half8(const uint16_t *p) { return *reinterpret_cast<const half8u_t *>(p); }
__device__ __forceinline__ void store_half8(uint16_t *p, half8_t v) { *reinterpret_cast<half8u_t *>(p) = v; }

// one output (row, col), its operands read here
__device__ __forceinline__ float epilogue_at(const Epilogue &e, float h, int row, int col, int N)
{
    const size_t at = (size_t)row * N + col;
    if (e.bias) h += (float)as_half(e.bias[col]);
    h = activate(h, e.act);
    if (e.mul) h *= (float)as_half(e.mul[at]);
    if (e.residual) h += (float)as_half(e.residual[at]);
    return h;
}

}  // namespace qmm
