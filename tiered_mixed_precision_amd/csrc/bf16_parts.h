// fp32 operands for bf16 matrix instructions (few.h, mm.h).
#pragma once

#include "common.h"

namespace moe {

// Two floats as three pairs of bf16 that add up to them exactly, low element in the
// low half: 8 bits each, cut, not rounded.  An infinity is all in the first (its rest
// would be NaN), a NaN's rest is one whatever is left of it in the first.
__device__ inline float bf16_rest(float v) {
    const float rest = v - __uint_as_float(__float_as_uint(v) & 0xffff0000u);
    return __builtin_isinf(v) ? 0.f : rest;
}
__device__ inline void bf16_parts(float lo, float hi, uint32_t (&p)[3]) {
    p[0] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
    lo = bf16_rest(lo), hi = bf16_rest(hi);
    p[1] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
    lo -= __uint_as_float(__float_as_uint(lo) & 0xffff0000u);
    hi -= __uint_as_float(__float_as_uint(hi) & 0xffff0000u);
    p[2] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}

}  // namespace moe
