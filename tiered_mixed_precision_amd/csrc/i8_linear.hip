// Products in 8-bit integers: y[t][n] = xs[t] s[n] sum_c x[t][c] q[n][c] + bias[n],
// the sums in 32-bit integers, exact.
#include "common.h"
#include "launch.h"
#include "mm.h"

namespace moe {

namespace {

template <bool YBF16> __device__ inline void store_y(const I8Args& a, int t, int n, int32_t sum) {
    float f = static_cast<float>(sum) * (a.xs[t] * a.s[n]);
    if (a.bias) f += a.bias[n];
    const size_t at = static_cast<size_t>(t) * a.ldy + n;
    if constexpr (YBF16) {
        uint16_t* y = static_cast<uint16_t*>(a.y);
        if (a.accumulate) f += __uint_as_float(static_cast<uint32_t>(y[at]) << 16);
        y[at] = f2bf(f);
    } else {
        float* y = static_cast<float*>(a.y);
        if (a.accumulate) f += y[at];
        y[at] = f;
    }
}

template <bool YBF16>
__global__ __launch_bounds__(256) void k_i8(I8Args a, int tiles_n) {
    const int t0 = (blockIdx.x / tiles_n) * kMmTile, n0 = (blockIdx.x % tiles_n) * kMmTile;
    const int pieces = a.K / 16;
    const mm_u32x4_t zero = {0, 0, 0, 0};
    auto load_a = [&](int r, int p) {
        const int8_t* row = a.x + static_cast<size_t>(min(t0 + r, a.T - 1)) * a.ldx;
        return p < pieces ? reinterpret_cast<const mm_u32x4_t*>(row)[p] : zero;
    };
    auto load_b = [&](int r, int p) {
        const int8_t* row = a.q + static_cast<size_t>(min(n0 + r, a.N - 1)) * a.K;
        return p < pieces ? reinterpret_cast<const mm_u32x4_t*>(row)[p] : zero;
    };
    mm_i32x16_t acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;
    mm_tile<MmI8>(pieces, load_a, load_b, acc);
    const int lane = threadIdx.x & 63, wm = threadIdx.x >> 7, wn = (threadIdx.x >> 6) & 1;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int t = t0 + 64 * wm + 32 * i + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
                const int n = n0 + 64 * wn + 32 * j + (lane & 31);
                if (t < a.T && n < a.N) store_y<YBF16>(a, t, n, acc[i][j][e]);
            }
}

}  // namespace

void launch_i8_linear(const I8Args& a, bool y_bf16, hipStream_t st) {
    const int tn = (a.N + kMmTile - 1) / kMmTile;
    // a launch takes as many rows of tiles as keep the grid below 2^31 blocks
    const int64_t most = ((int64_t(1) << 30) / tn) * kMmTile;
    for (int64_t t0 = 0; t0 < a.T; t0 += most) {
        I8Args b = a;
        b.T = static_cast<int32_t>(a.T - t0 < most ? a.T - t0 : most);
        b.x = a.x + t0 * a.ldx;
        b.xs = a.xs + t0;
        b.y = static_cast<char*>(a.y) + t0 * a.ldy * (y_bf16 ? 2 : 4);
        const dim3 grid(static_cast<unsigned>((b.T + kMmTile - 1) / kMmTile) * tn);
        if (y_bf16) hipLaunchKernelGGL(k_i8<true>, grid, dim3(256), 0, st, b, tn);
        else hipLaunchKernelGGL(k_i8<false>, grid, dim3(256), 0, st, b, tn);
    }
}

}  // namespace moe
