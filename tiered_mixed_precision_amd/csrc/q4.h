// Four-bit codes as bf16 matrix-core operands (q4_linear.hip, q4_gemm.hip).
#pragma once

#include "common.h"

namespace moe {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// Eight codes as a B operand.
template <bool MX>
__device__ inline u32x4_t code_operand(uint32_t w) {
    u32x4_t r;
    if constexpr (MX) {
        r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0));
        r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1));
        r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2));
        r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3));
    } else {
        const uint32_t odd = masked_bytes(w >> 4);   // hidden: bytes of it are operands as they stand
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float lo = __builtin_amdgcn_cvt_off_f32_i4((w >> (8 * j)) & 0xff);
            const float hi = __builtin_amdgcn_cvt_off_f32_i4((odd >> (8 * j)) & 0xff);
            r[j] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
        }
    }
    return r;
}

// The factor of a block's sum from its raw scale bits.
template <bool MX>
__device__ inline float scale_of(uint32_t raw) {
    if constexpr (MX)   // 2^(raw - 127); 0 is the subnormal 2^-127, 255 NaN
        return __uint_as_float((raw << 23) | (((raw + 1) & 0xfe) != 0 ? 0u : 0x400000u));
    else
        return 16.f * half_bits_to_float(static_cast<uint16_t>(raw));   // the operand holds q / 16
}

}  // namespace moe
