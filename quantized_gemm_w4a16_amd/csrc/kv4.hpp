// kv4.hpp -- what the cache of 4 bits, its write and the attention over it share.
#pragma once

#include "spear_internal.hpp"

namespace spear {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// Eight codes of one block as bf16, in order: a conversion an output pair, exact
// (an e2m1 level times a power of two).  A scale of infinity (byte 255) gives NaN.
__device__ __forceinline__ u32x4 kv4_bf16(uint32_t codes, float scale)
{
    u32x4 r;
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3));
    return r;
}

// The scale byte as the power of two.
__device__ __forceinline__ float kv4_scale(uint32_t byte) { return __uint_as_float(byte << 23); }

// Two fp32 to a pair of bf16 in one instruction.
__device__ __forceinline__ uint32_t pair_bf16(float lo, float hi)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

// Host: SPEAR_OK if the cache's pointers and sizes are as spear.h has them.
spear_status check_kv4(const spear_kv4 *kv);

} // namespace spear
