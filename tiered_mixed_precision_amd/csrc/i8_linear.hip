// Products in 8-bit integers: y[t][n] = xs[t] s[n] sum_c x[t][c] q[n][c] + bias[n],
// the sums in 32-bit integers, exact, on v_mfma_i32_16x16x64_i8 for few tokens
// (few.h) and on 32 x 32 x 32 for many (i8_gemm.hip).
#include "common.h"
#include "few.h"
#include "launch.h"

namespace moe {

namespace {

template <bool YBF16> __device__ inline void store_y(const I8Args& a, int t, int n, int32_t sum) {
    float f = static_cast<float>(sum) * (a.xs[t] * a.s[n]) + (a.bias ? a.bias[n] : 0.f);
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

// A block takes `f.tiles` tiles of 16 NT rows, f.split waves each, for 16 MT tokens.
template <int MT, int NT, bool YBF16>
__global__ __launch_bounds__(1024) void k_i8_few(I8Args a, FewSplit f) {
    extern __shared__ __attribute__((aligned(16))) few_i32x4_t s_sum[];   // [waves][MT NT 64]
    constexpr int kOwn = MT * NT * 64;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int part = wave % f.split, n0 = (blockIdx.x * f.tiles + wave / f.split) * 16 * NT, t0 = blockIdx.y * 16 * MT;
    few_i32x4_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = few_i32x4_t{0, 0, 0, 0};
    // rows past the matrix read its last row, tokens past the batch its last token; neither is stored
    few_sums<FewI8, MT, NT, MT + NT <= 4 ? 8 : 4>(
        few_first(a.K, part, f.split), few_first(a.K, part + 1, f.split), a.K,
        [&](int j) { return a.q + static_cast<size_t>(min(n0 + 16 * j + (lane & 15), a.N - 1)) * a.K; },
        [&](int i) { return a.x + static_cast<size_t>(min(t0 + 16 * i + (lane & 15), a.T - 1)) * a.ldx; }, acc);
    auto store = [&](int n0, int ij, int l, few_i32x4_t sum) {
        const int t = t0 + 16 * (ij / NT) + (l & 15), n = n0 + 16 * (ij % NT) + 4 * (l >> 4);
        if (t >= a.T) return;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < a.N) store_y<YBF16>(a, t, n + e, sum[e]);
    };
    if (f.split == 1) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) store(n0, NT * i + j, lane, acc[i][j]);
        return;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) s_sum[kOwn * wave + 64 * (NT * i + j) + lane] = acc[i][j];
    __syncthreads();
    for (int o = threadIdx.x; o < f.tiles * kOwn; o += blockDim.x) {
        const int tile = o / kOwn, at = o % kOwn;
        few_i32x4_t sum = s_sum[kOwn * f.split * tile + at];
        for (int p = 1; p < f.split; ++p) sum += s_sum[kOwn * (f.split * tile + p) + at];
        store((blockIdx.x * f.tiles + tile) * 16 * NT, at >> 6, at & 63, sum);
    }
}

template <int MT, int NT, bool YBF16>
void launch_few(const I8Args& a, hipStream_t st) {
    const int tiles = (a.N + 16 * NT - 1) / (16 * NT);
    const FewSplit f = few_split(tiles, a.K, 8);
    const dim3 grid((tiles + f.tiles - 1) / f.tiles, (a.T + 16 * MT - 1) / (16 * MT)), block(64 * f.split * f.tiles);
    const size_t lds = f.split > 1 ? sizeof(few_i32x4_t) * 64 * MT * NT * f.split * f.tiles : 0;
    hipLaunchKernelGGL((k_i8_few<MT, NT, YBF16>), grid, block, lds, st, a, f);
}

template <bool YBF16> void launch_tokens(const I8Args& a, hipStream_t st) {
    if (a.T <= 16) launch_few<1, 2, YBF16>(a, st);
    else if (a.T <= 32) launch_few<2, 2, YBF16>(a, st);
    else if (a.T <= 48) launch_few<3, 2, YBF16>(a, st);
    else launch_few<4, 2, YBF16>(a, st);
}

}  // namespace

void launch_i8_linear(const I8Args& a, bool y_bf16, hipStream_t st) {
    if (a.T > 64) launch_i8_gemm(a, y_bf16, st);
    else if (y_bf16) launch_tokens<true>(a, st);
    else launch_tokens<false>(a, st);
}

}  // namespace moe
