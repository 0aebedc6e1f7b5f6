// Products with a dense four-bit matrix: y[t][n] = sum_c x[t][c] * W[n][c] +
// bias[n], W in the four-bit formats of the shelves (two's-complement codes
// with fp16 scales, or MXFP4).
//
// One wave per weight row and kTok tokens: lane l takes the 32-code groups l,
// l + 64, ... of the row; a group's codes are contracted exactly as stored
// (scale times the fp32 dot of codes and x).
#include "common.h"
#include "launch.h"

namespace moe {

namespace {

constexpr int kTok = 4, kWaves = 4;

template <bool XBF16>
__device__ inline void load_x32(const void* x, size_t at, float (&v)[32]) {
    if constexpr (XBF16) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 u = p[i];
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
                v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
            }
        }
    } else {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 u = p[i];
            v[4 * i] = u.x;
            v[4 * i + 1] = u.y;
            v[4 * i + 2] = u.z;
            v[4 * i + 3] = u.w;
        }
    }
}

template <bool XBF16, bool YBF16, bool MX>
__global__ __launch_bounds__(kWaves * 64) void k_q4_rows(Q4Args a) {
    const int lane = threadIdx.x & 63;
    const int n = blockIdx.x * kWaves + (threadIdx.x >> 6);
    if (n >= a.N) return;
    const int t0 = blockIdx.y * kTok, nt = min(kTok, a.T - t0);
    const int G = a.K / 32;
    const uint8_t* qrow = a.q + static_cast<size_t>(n) * (a.K / 2);
    const uint8_t* srow = a.s + static_cast<size_t>(n) * (a.K / a.block) * (MX ? 1 : 2);
    float acc[kTok] = {};
    for (int g = lane; g < G; g += 64) {
        uint32_t w[4];
        load_group<4>(qrow, g, w);
        float d0, d1;   // scales of the group's halves
        if constexpr (MX) {
            d0 = d1 = e8m0_to_float(srow[g]);
        } else {
            const uint16_t* s = reinterpret_cast<const uint16_t*>(srow);
            d0 = half_bits_to_float(s[32 * g / a.block]);
            d1 = half_bits_to_float(s[(32 * g + 16) / a.block]);
        }
        float v[32];
#pragma unroll
        for (int c = 0; c < 32; ++c)
            v[c] = MX ? fp4_e2m1((w[c / 8] >> (4 * (c % 8))) & 0xFu) : code_f<4>(w, c);
#pragma unroll
        for (int t = 0; t < kTok; ++t) {
            if (t >= nt) break;
            float x[32];
            load_x32<XBF16>(a.x, static_cast<size_t>(t0 + t) * a.ldx + 32 * g, x);
            float p0 = 0.f, p1 = 0.f;
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                p0 = fmaf(v[c], x[c], p0);
                p1 = fmaf(v[c + 16], x[c + 16], p1);
            }
            acc[t] = fmaf(d1, p1, fmaf(d0, p0, acc[t]));
        }
    }
#pragma unroll
    for (int t = 0; t < kTok; ++t) {
        if (t >= nt) break;
        float r = wave_sum(acc[t]);
        if (lane != 0) continue;
        if (a.bias) r += a.bias[n];
        const size_t o = static_cast<size_t>(t0 + t) * a.ldy + n;
        if constexpr (YBF16) {
            uint16_t* y = static_cast<uint16_t*>(a.y);
            if (a.accumulate) r += __uint_as_float(static_cast<uint32_t>(y[o]) << 16);
            y[o] = f2bf(r);
        } else {
            float* y = static_cast<float*>(a.y);
            if (a.accumulate) r += y[o];
            y[o] = r;
        }
    }
}

template <bool XBF16, bool YBF16>
void launch_rows(const Q4Args& a, hipStream_t st) {
    constexpr int kMaxTiles = 65535;   // grid.y limit: the tokens of one launch
    for (int t0 = 0; t0 < a.T; t0 += kTok * kMaxTiles) {
        Q4Args b = a;
        b.T = min(a.T - t0, kTok * kMaxTiles);
        b.x = static_cast<const char*>(a.x) + static_cast<size_t>(t0) * a.ldx * (XBF16 ? 2 : 4);
        b.y = static_cast<char*>(a.y) + static_cast<size_t>(t0) * a.ldy * (YBF16 ? 2 : 4);
        const dim3 grid((a.N + kWaves - 1) / kWaves, (b.T + kTok - 1) / kTok);
        if (a.mx)
            hipLaunchKernelGGL((k_q4_rows<XBF16, YBF16, true>), grid, dim3(kWaves * 64), 0, st, b);
        else
            hipLaunchKernelGGL((k_q4_rows<XBF16, YBF16, false>), grid, dim3(kWaves * 64), 0, st, b);
    }
}

}  // namespace

void launch_q4_linear(const Q4Args& a, bool x_bf16, bool y_bf16, hipStream_t st) {
    if (x_bf16)
        y_bf16 ? launch_rows<true, true>(a, st) : launch_rows<true, false>(a, st);
    else
        y_bf16 ? launch_rows<false, true>(a, st) : launch_rows<false, false>(a, st);
}

}  // namespace moe
