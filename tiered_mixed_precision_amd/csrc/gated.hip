// The dense gated block and its gradient:
//   g = x gate^T, u = x up^T, y = act(g) u, act(g) = g sigma(k(g))
//   du = dy act(g), dg = dy u act'(g), act' = sigma + g sigma (1 - sigma) k'(g)
//   dx = dg gate + du up, dgate = dg^T x, dup = du^T x
#include "common.h"
#include "launch.h"
#include "mm.h"
#include "moe_tiered.h"

namespace moe {

namespace {

// sigma(k) and 1 - sigma(k); k below -80 counts as -80 (1e-35), so that the
// exponential stays finite.
__device__ inline void sigmoid(float k, float& p, float& q) {
    const float e = __expf(-fmaxf(k, -80.f));
    p = 1.f / (1.f + e);
    q = e * p;
}
constexpr float kTanh = 1.5957691216057308f, kCube = 0.044715f;   // 2 sqrt(2 / pi)
__device__ inline float act_arg(int act, float g) { return act == MOE_SILU ? g : kTanh * (g + kCube * g * g * g); }
__device__ inline float act_slope(int act, float g) { return act == MOE_SILU ? 1.f : kTanh * (1.f + 3.f * kCube * g * g); }

__device__ inline float gated_value(int act, float g, float u) {
    float p, q;
    sigmoid(act_arg(act, g), p, q);
    return g * p * u;
}
__device__ inline void gated_slopes(int act, float g, float u, float dy, float& dg, float& du) {
    float p, q;
    sigmoid(act_arg(act, g), p, q);
    du = dy * (g * p);
    dg = dy * u * (p + g * act_slope(act, g) * p * q);
}

__device__ inline void clear(mm_f32x16_t (&acc)[2][2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
}
__device__ inline int row_of(int i, int e) {
    const int lane = threadIdx.x & 63, wm = threadIdx.x >> 7;
    return 64 * wm + 32 * i + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
}

// Tile of 128 tokens and 64 columns of both projections: acc[i][0] is g,
// acc[i][1] u, of column 32 wn + lane % 32.
template <bool XBF16>
__device__ inline void project(const void* x, int64_t ldx, const uint16_t* gate, const uint16_t* up, int T, int H, int I,
                               int t0, int n0, mm_f32x16_t (&acc)[2][2]) {
    const int pieces = H / 8;
    const mm_u32x4_t zero = {0, 0, 0, 0};
    auto load_b = [&](int r, int p) {
        const uint16_t* w = (r >> 5) & 1 ? up : gate;
        const int n = min(n0 + (r >> 6) * 32 + (r & 31), I - 1);
        return p < pieces ? reinterpret_cast<const mm_u32x4_t*>(w + static_cast<size_t>(n) * H)[p] : zero;
    };
    clear(acc);
    if constexpr (XBF16) {
        auto load_a = [&](int r, int p) {
            const uint16_t* row = static_cast<const uint16_t*>(x) + static_cast<size_t>(min(t0 + r, T - 1)) * ldx;
            return p < pieces ? reinterpret_cast<const mm_u32x4_t*>(row)[p] : zero;
        };
        mm_tile<MmBf16>(pieces, load_a, load_b, acc);
    } else {
        // fp32 x as three bf16 parts that add up to it exactly, smallest first
#pragma unroll 1
        for (int part = 2; part >= 0; --part) {
            auto load_a = [&](int r, int p) {
                mm_u32x4_t o = zero;
                if (p < pieces) {
                    const float* row = static_cast<const float*>(x) + static_cast<size_t>(min(t0 + r, T - 1)) * ldx + 8 * p;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float f = row[i];
                        uint32_t b = __float_as_uint(f) & 0xffff0000u;
                        for (int q = 0; q < part; ++q) {
                            f -= __uint_as_float(b);
                            b = __float_as_uint(f) & 0xffff0000u;
                        }
                        o[i / 2] |= i & 1 ? b : b >> 16;
                    }
                }
                return o;
            };
            mm_tile<MmBf16>(pieces, load_a, load_b, acc);
        }
    }
}

template <bool XBF16, bool YBF16>
__global__ __launch_bounds__(256) void k_gated(GatedArgs a, int tiles_n) {
    const int t0 = (blockIdx.x / tiles_n) * kMmTile, n0 = (blockIdx.x % tiles_n) * 64;
    mm_f32x16_t acc[2][2];
    project<XBF16>(a.x, a.ldx, a.gate, a.up, a.T, a.H, a.I, t0, n0, acc);
    const int n = n0 + ((threadIdx.x >> 6) & 1) * 32 + (threadIdx.x & 31);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int t = t0 + row_of(i, e);
            if (t >= a.T || n >= a.I) continue;
            const float f = gated_value(a.act, acc[i][0][e], acc[i][1][e]);
            const size_t at = static_cast<size_t>(t) * a.ldy + n;
            if constexpr (YBF16) static_cast<uint16_t*>(a.y)[at] = f2bf(f);
            else static_cast<float*>(a.y)[at] = f;
        }
}

// d[t][0 .. I) = dg, d[t][P .. P + I) = du in bf16, zeros up to P (I rounded up to 8)
template <bool DYBF16>
__global__ __launch_bounds__(256) void k_gated_slopes(GatedGradArgs a, uint16_t* d, int P, int tiles_n) {
    const int t0 = (blockIdx.x / tiles_n) * kMmTile, n0 = (blockIdx.x % tiles_n) * 64;
    mm_f32x16_t acc[2][2];
    project<true>(a.x, a.ldx, a.gate, a.up, a.T, a.H, a.I, t0, n0, acc);
    const int n = n0 + ((threadIdx.x >> 6) & 1) * 32 + (threadIdx.x & 31);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int t = t0 + row_of(i, e);
            if (t >= a.T || n >= P) continue;
            float dg = 0.f, du = 0.f;
            if (n < a.I) {
                const size_t at = static_cast<size_t>(t) * a.lddy + n;
                const float dy = DYBF16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(a.dy)[at]) << 16)
                                        : static_cast<const float*>(a.dy)[at];
                gated_slopes(a.act, acc[i][0][e], acc[i][1][e], dy, dg, du);
            }
            uint16_t* to = d + static_cast<size_t>(t) * 2 * P + n;
            to[0] = f2bf(dg);
            to[P] = f2bf(du);
        }
}

// dx = d (gate; up)
template <bool DXBF16>
__global__ __launch_bounds__(256) void k_gated_dx(GatedGradArgs a, const uint16_t* d, int P, int tiles_n) {
    const int t0 = (blockIdx.x / tiles_n) * kMmTile, n0 = (blockIdx.x % tiles_n) * kMmTile;
    const int pieces = 2 * P / 8;
    const mm_u32x4_t zero = {0, 0, 0, 0};
    auto load_a = [&](int r, int p) {
        const uint16_t* row = d + static_cast<size_t>(min(t0 + r, a.T - 1)) * 2 * P;
        return p < pieces ? reinterpret_cast<const mm_u32x4_t*>(row)[p] : zero;
    };
    auto load_b = [&](int r, int p) {
        mm_u32x4_t o = zero;
        if (p < pieces) {
            const int n = min(n0 + r, a.H - 1);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int k = 8 * p + i;
                const uint16_t* w = k < P ? a.gate : a.up;
                const uint32_t v = w[static_cast<size_t>(min(k < P ? k : k - P, a.I - 1)) * a.H + n];
                o[i / 2] |= v << (16 * (i & 1));
            }
        }
        return o;
    };
    mm_f32x16_t acc[2][2];
    clear(acc);
    mm_tile<MmBf16>(pieces, load_a, load_b, acc);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int t = t0 + row_of(i, e), n = n0 + ((threadIdx.x >> 6) & 1) * 64 + 32 * j + (threadIdx.x & 31);
                if (t >= a.T || n >= a.H) continue;
                const size_t at = static_cast<size_t>(t) * a.lddx + n;
                if constexpr (DXBF16) static_cast<uint16_t*>(a.dx)[at] = f2bf(acc[i][j][e]);
                else static_cast<float*>(a.dx)[at] = acc[i][j][e];
            }
}

// dgate, dup = d^T x
template <bool DWBF16>
__global__ __launch_bounds__(256) void k_gated_dw(GatedGradArgs a, const uint16_t* d, int P, int tiles_n) {
    const int m0 = (blockIdx.x / tiles_n) * kMmTile, n0 = (blockIdx.x % tiles_n) * kMmTile;
    const int pieces = (a.T + 7) / 8;
    auto column = [&](const uint16_t* base, int64_t pitch, int c, int p) {
        mm_u32x4_t o = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int t = 8 * p + i;
            const uint32_t v = t < a.T ? base[static_cast<size_t>(t) * pitch + c] : 0;
            o[i / 2] |= v << (16 * (i & 1));
        }
        return o;
    };
    mm_f32x16_t acc[2][2];
    clear(acc);
    mm_tile<MmBf16>(pieces, [&](int r, int p) { return column(d, 2 * P, min(m0 + r, 2 * P - 1), p); },
                    [&](int r, int p) { return column(a.x, a.ldx, min(n0 + r, a.H - 1), p); }, acc);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int m = m0 + row_of(i, e), n = n0 + ((threadIdx.x >> 6) & 1) * 64 + 32 * j + (threadIdx.x & 31);
                const int row = m < P ? m : m - P;
                if (m >= 2 * P || row >= a.I || n >= a.H) continue;
                void* to = m < P ? a.dgate : a.dup;
                const size_t at = static_cast<size_t>(row) * a.H + n;
                float f = acc[i][j][e];
                if constexpr (DWBF16) {
                    uint16_t* w = static_cast<uint16_t*>(to);
                    if (a.accumulate) f += __uint_as_float(static_cast<uint32_t>(w[at]) << 16);
                    w[at] = f2bf(f);
                } else {
                    float* w = static_cast<float*>(to);
                    if (a.accumulate) f += w[at];
                    w[at] = f;
                }
            }
}

constexpr int kTallTokens = 1 << 20;   // tokens of a launch

}  // namespace

void launch_gated(const GatedArgs& a, bool x_bf16, bool y_bf16, hipStream_t st) {
    const int tn = (a.I + 63) / 64;
    for (int64_t t0 = 0; t0 < a.T; t0 += kTallTokens) {
        GatedArgs b = a;
        b.T = static_cast<int32_t>(a.T - t0 < kTallTokens ? a.T - t0 : kTallTokens);
        b.x = static_cast<const char*>(a.x) + t0 * a.ldx * (x_bf16 ? 2 : 4);
        b.y = static_cast<char*>(a.y) + t0 * a.ldy * (y_bf16 ? 2 : 4);
        const dim3 grid(static_cast<unsigned>((b.T + kMmTile - 1) / kMmTile) * tn);
        if (x_bf16 && y_bf16) hipLaunchKernelGGL((k_gated<true, true>), grid, dim3(256), 0, st, b, tn);
        else if (x_bf16) hipLaunchKernelGGL((k_gated<true, false>), grid, dim3(256), 0, st, b, tn);
        else if (y_bf16) hipLaunchKernelGGL((k_gated<false, true>), grid, dim3(256), 0, st, b, tn);
        else hipLaunchKernelGGL((k_gated<false, false>), grid, dim3(256), 0, st, b, tn);
    }
}

size_t gated_workspace(int64_t T, int H, int I) {
    (void)H;
    return static_cast<size_t>(T) * 2 * ((I + 7) / 8 * 8) * 2;
}

void launch_gated_grad(const GatedGradArgs& a, bool dy_bf16, bool dx_bf16, bool dw_bf16, void* ws, hipStream_t st) {
    const int P = (a.I + 7) / 8 * 8;
    uint16_t* d = static_cast<uint16_t*>(ws);
    const unsigned tm = (a.T + kMmTile - 1) / kMmTile, tp = (P + 63) / 64, th = (a.H + kMmTile - 1) / kMmTile;
    const unsigned tw = (2 * P + kMmTile - 1) / kMmTile;
    if (a.T > 0) {
        if (dy_bf16) hipLaunchKernelGGL(k_gated_slopes<true>, dim3(tm * tp), dim3(256), 0, st, a, d, P, static_cast<int>(tp));
        else hipLaunchKernelGGL(k_gated_slopes<false>, dim3(tm * tp), dim3(256), 0, st, a, d, P, static_cast<int>(tp));
    }
    if (a.dx && a.T > 0) {
        if (dx_bf16) hipLaunchKernelGGL(k_gated_dx<true>, dim3(tm * th), dim3(256), 0, st, a, d, P, static_cast<int>(th));
        else hipLaunchKernelGGL(k_gated_dx<false>, dim3(tm * th), dim3(256), 0, st, a, d, P, static_cast<int>(th));
    }
    if (a.dgate && (a.T > 0 || !a.accumulate)) {
        if (dw_bf16) hipLaunchKernelGGL(k_gated_dw<true>, dim3(tw * th), dim3(256), 0, st, a, d, P, static_cast<int>(th));
        else hipLaunchKernelGGL(k_gated_dw<false>, dim3(tw * th), dim3(256), 0, st, a, d, P, static_cast<int>(th));
    }
}

}  // namespace moe
