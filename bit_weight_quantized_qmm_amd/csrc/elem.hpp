// elem.hpp -- element types of activations and caches, and their conversions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmm {

typedef __bf16 bf16_t;
struct fp8_t { uint8_t b; };   // e4m3 (OCP: 4 exponent bits, bias 7, largest 448, no infinity)

__device__ __forceinline__ float to_f32(_Float16 x) { return (float)x; }
__device__ __forceinline__ float to_f32(bf16_t x) { return (float)x; }

// fp32 -> element, ties to even; e4m3 saturates at +-448 and keeps NaN
template <typename S> __device__ __forceinline__ S from_f32(float x) { return (S)x; }
template <> __device__ __forceinline__ fp8_t from_f32<fp8_t>(float x)
{
    x = x > 448.f ? 448.f : x < -448.f ? -448.f : x;   // NaN passes both comparisons unchanged
    return fp8_t{(uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(x, x, 0, false) & 0xff)};
}

}  // namespace qmm
