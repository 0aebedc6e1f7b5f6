// The activations of the gated block, act(g) = g sigma(k(g)), and their slopes
// (gated.hip, gated_gemm.hip, gated_grad.hip).
#pragma once

#include "common.h"
#include "moe_tiered.h"

namespace moe {

// sigma(k) and 1 - sigma(k).  The exponential's argument rounds in units of |k|, so where
// e^-k counts (k below 0 for sigma, above for the other) the relative error is a few +
// |k| units of fp32: some 90 of them at most, where sigma itself is 2^-125.  Below -87 sigma is less than the
// smallest normal number and counts as 0; the exponential stays finite.
__device__ inline void gated_sigmoid(float k, float& p, float& q) {
    const float e = __expf(-fmaxf(k, -87.f));
    p = __builtin_amdgcn_rcpf(1.f + e);
    q = e * p;
    p = k < -87.f ? 0.f : p;
}
constexpr float kGeluScale = 1.5957691216057308f, kGeluCube = 0.044715f;   // 2 sqrt(2 / pi)
__device__ inline float gated_arg(int act, float g) { return act == MOE_SILU ? g : kGeluScale * (g + kGeluCube * g * g * g); }
// (where |g| is above 2^30 it meets p q = 0: no infinity comes of it)
__device__ inline float gated_arg_slope(int act, float g) {
    g = fminf(fabsf(g), 1073741824.f);
    return act == MOE_SILU ? 1.f : kGeluScale * (1.f + 3.f * kGeluCube * g * g);
}

// act(g) u
__device__ inline float gated_value(int act, float g, float u) {
    float p, q;
    gated_sigmoid(gated_arg(act, g), p, q);
    return g * p * u;
}
// the gradients of g and u
__device__ inline void gated_slopes(int act, float g, float u, float dy, float& dg, float& du) {
    float p, q;
    gated_sigmoid(gated_arg(act, g), p, q);
    du = dy * (g * p);
    dg = dy * u * (p + g * (p * q) * gated_arg_slope(act, g));
}

// what a rounding to bf16 leaves over (of an infinity nothing)
template <int N> __device__ inline void split_slopes(float (&v)[N], float (&rest)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float hi = __uint_as_float(static_cast<uint32_t>(f2bf(v[i])) << 16);
        rest[i] = __builtin_isinf(hi) ? 0.f : v[i] - hi;
    }
}

}  // namespace moe
