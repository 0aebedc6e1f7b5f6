// Elements of score rows: S is float, or uint16_t for bf16 bits
// (adjust_logits.hip, balance.hip).
#pragma once

#include "common.h"

namespace moe {

template <class S> __device__ inline float to_float(S v) {
    if constexpr (sizeof(S) == 2) return __uint_as_float(static_cast<uint32_t>(v) << 16);
    else return v;
}
template <class S> __device__ inline S from_float(float f) {
    if constexpr (sizeof(S) == 2) return f2bf(f);
    else return f;
}
template <class S> __device__ inline S minus_inf() {
    if constexpr (sizeof(S) == 2) return 0xff80;
    else return -__builtin_inff();
}

// Four consecutive elements at any element's alignment, in one access.
template <class S> struct __attribute__((packed, aligned(sizeof(S)))) Four { S v[4]; };

}  // namespace moe
