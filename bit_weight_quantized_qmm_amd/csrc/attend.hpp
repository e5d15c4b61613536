// attend.hpp -- what the attention kernels share: operand types, the matrix instructions
// of either element type, and the pages of a sequence.
#pragma once

#include "elem.hpp"
#include "launch.hpp"
#include "qmm_device.hpp"

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

template <typename A>
__device__ __forceinline__ int key_page(const A &a, int key)
{
    return (int)(((uint64_t)(uint32_t)key * a.page_mul) >> a.page_sh);
}

// Whether one of the keys [lo, hi) of sequence b stands on a page of the cache.
// Asked of rows without a sum alone.
template <typename A>
__device__ __forceinline__ bool sees_key(const A &a, int b, int64_t lo, int64_t hi)
{
    for (int64_t key = lo > 0 ? lo : 0; key < hi;) {
        const int pg = key_page(a, (int)key);
        if ((uint32_t)a.table[b * a.table_s + pg] < (uint32_t)a.pages) return true;
        key = ((int64_t)pg + 1) * a.page;
    }
    return false;
}

}  // namespace qmm
