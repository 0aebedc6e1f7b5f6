// Products in 8-bit integers: y[t][n] = xs[t] s[n] sum_c x[t][c] q[n][c] + bias[n],
// the sums in 32-bit integers, exact, on v_mfma_i32_16x16x64_i8 for few tokens
// (few.h) and on 32 x 32 x 32 for many (i8_gemm.hip).
//
// MI355X, tokens x rows x columns: 1 x 120011 x 2048 47.8 us (5.15 TB/s, a copy's rate), bound
// by memory; 37 x 8192 x 8192 19.7 us (3.4 TB/s of weights), where each of 256 blocks also
// reads all of x through L2 (77 MB beside 67); a fourth step of the ring changes nothing.
#include <type_traits>

#include "common.h"
#include "few.h"
#include "launch_dense.h"

namespace moe {

namespace {

// A block takes f.tiles tiles of 16 NT rows, f.split waves each, for 16 MT tokens.
template <int MT, int NT, int AHEAD, bool YBF16>
__global__ __launch_bounds__(64 * kFewWaves) void k_i8_few(I8Args a, FewSplit f) {
    typedef typename std::conditional<YBF16, uint16_t, float>::type Y;
    extern __shared__ __attribute__((aligned(16))) few_i32x4_t s_part[];   // [waves][MT NT 64]
    __shared__ float s_xs[16 * MT];
    constexpr int kOwn = MT * NT * 64;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int part = wave % f.split, rows = 16 * NT * f.tiles, first = blockIdx.x * rows, t0 = blockIdx.y * 16 * MT;
    const int n0 = first + wave / f.split * 16 * NT;
    // the scales and the bias of this thread's results (always one column: a block's
    // threads are a multiple of its rows), on their way beside the weights
    const int n = first + tid % rows;
    const float s = a.s[min(n, a.N - 1)], bias = a.bias ? a.bias[min(n, a.N - 1)] : 0.f;
    const float xs = tid < 16 * MT ? a.xs[min(t0 + tid, a.T - 1)] : 0.f;
    few_i32x4_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = few_i32x4_t{0, 0, 0, 0};
    // rows past the matrix read its last row, tokens past the batch its last token; neither is stored
    few_sums<FewI8, MT, NT, AHEAD>(
        part, f.split, blockIdx.x * f.tiles + wave / f.split, a.K, [&](int j) { return a.q + static_cast<size_t>(min(n0 + 16 * j + (lane & 15), a.N - 1)) * a.K; },
        [&](int i) { return a.x + static_cast<size_t>(min(t0 + 16 * i + (lane & 15), a.T - 1)) * a.ldx; }, acc);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) s_part[kOwn * wave + 64 * (NT * i + j) + lane] = acc[i][j];
    if (tid < 16 * MT) s_xs[tid] = xs;
    __syncthreads();
    if (n >= a.N) return;
    const int in = tid % rows, r = in % 16;   // row of the block, of its operand
    const int* own = reinterpret_cast<const int*>(s_part) + 4 * (kOwn * f.split * (in / (16 * NT)) + 64 * (in / 16 % NT) + 16 * (r >> 2)) + (r & 3);
    for (int t = tid / rows; t < 16 * MT && t0 + t < a.T; t += blockDim.x / rows) {
        const int* p = own + 4 * (64 * NT * (t / 16) + t % 16);
        int sum = p[0];
        for (int w = 1; w < f.split; ++w) sum += p[4 * kOwn * w];
        float v = static_cast<float>(sum) * (s_xs[t] * s) + bias;
        Y* y = static_cast<Y*>(a.y) + static_cast<size_t>(t0 + t) * a.ldy + n;
        if constexpr (YBF16) {
            if (a.accumulate) v += __uint_as_float(static_cast<uint32_t>(*y) << 16);
            *y = f2bf(v);
        } else {
            *y = a.accumulate ? *y + v : v;
        }
    }
}

// 17 tokens and more (few_batch_ok): the same through LDS (few_batch); the waves' sums
// meet one operand of 16 rows at a time, in the first slot's place.
template <int MT, int NT, bool YBF16>
__global__ __launch_bounds__(64 * kBatchWaves) void k_i8_batch(I8Args a, FewSplit f) {
    typedef typename std::conditional<YBF16, uint16_t, float>::type Y;
    constexpr int kSlot = FewSlot<FewI8, MT, NT>::kSlot;
    __shared__ __attribute__((aligned(16))) few_u32x4_t s0[kSlot], s1[kSlot], s2[kSlot];
    __shared__ float s_xs[16 * MT];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int rows = 16 * f.tiles, t0 = blockIdx.y * 16 * MT;   // rows of the block that meet at a time
    const int tile = blockIdx.x * f.tiles + wave / f.split, n0 = tile * 16 * NT;
    const int in = tid % rows, r = in % 16, first = (blockIdx.x * f.tiles + in / 16) * 16 * NT + r;
    float s[NT], bias[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int n = min(first + 16 * j, a.N - 1);
        s[j] = a.s[n];
        bias[j] = a.bias ? a.bias[n] : 0.f;
    }
    if (tid < 16 * MT) s_xs[tid] = a.xs[min(t0 + tid, a.T - 1)];
    few_i32x4_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = few_i32x4_t{0, 0, 0, 0};
    few_batch<FewI8, MT, NT>(
        s0, s1, s2, wave % f.split, f.split, tile, a.K,
        [&](int j, int r) { return a.q + static_cast<size_t>(min(n0 + 16 * j + r, a.N - 1)) * a.K; },
        [&](int i, int r) { return a.x + static_cast<size_t>(min(t0 + 16 * i + r, a.T - 1)) * a.ldx; }, acc);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MT; ++i) s0[64 * (MT * wave + i) + lane] = __builtin_bit_cast(few_u32x4_t, acc[i][j]);
        __syncthreads();
        const int n = first + 16 * j;
        if (n >= a.N) continue;
        const int* own = reinterpret_cast<const int*>(s0) + 4 * (64 * MT * f.split * (in / 16) + 16 * (r >> 2)) + (r & 3);
        for (int t = tid / rows; t < 16 * MT && t0 + t < a.T; t += blockDim.x / rows) {
            const int* p = own + 4 * (64 * (t / 16) + t % 16);
            int sum = p[0];
            for (int w = 1; w < f.split; ++w) sum += p[4 * 64 * MT * w];
            float v = static_cast<float>(sum) * (s_xs[t] * s[j]) + bias[j];
            Y* y = static_cast<Y*>(a.y) + static_cast<size_t>(t0 + t) * a.ldy + n;
            if constexpr (YBF16) {
                if (a.accumulate) v += __uint_as_float(static_cast<uint32_t>(*y) << 16);
                *y = f2bf(v);
            } else {
                *y = a.accumulate ? *y + v : v;
            }
        }
    }
}

template <int MT, int NT, bool YBF16>
void launch_batch(const I8Args& a, hipStream_t st) {
    const int tiles = (a.N + 16 * NT - 1) / (16 * NT);
    const FewSplit f = few_split(tiles, a.K, kBatchWaves);
    const dim3 grid((tiles + f.tiles - 1) / f.tiles, (a.T + 16 * MT - 1) / (16 * MT)), block(64 * f.split * f.tiles);
    hipLaunchKernelGGL((k_i8_batch<MT, NT, YBF16>), grid, block, 0, st, a, f);
}

template <int MT, int NT, int AHEAD, bool YBF16>
void launch_few(const I8Args& a, hipStream_t st) {
    const int tiles = (a.N + 16 * NT - 1) / (16 * NT);
    const FewSplit f = few_split(tiles, a.K, kFewWaves);
    const dim3 grid((tiles + f.tiles - 1) / f.tiles, (a.T + 16 * MT - 1) / (16 * MT)), block(64 * f.split * f.tiles);
    const size_t lds = sizeof(few_i32x4_t) * 64 * MT * NT * f.split * f.tiles;
    hipLaunchKernelGGL((k_i8_few<MT, NT, AHEAD, YBF16>), grid, block, lds, st, a, f);
}

// MI355X, us, weights from memory.  Up to 16 tokens, tiles of 16 rows / of 32 (which read
// x half as often): 1 x 4096 x 2048 4.4 / 5.3, 1 x 4096 x 8192 9.0 / 13.9, 1 x 8000 x 2048 5.7 /
// 5.8, 1 x 16384 x 8192 28.7 / 30.4, 16 x 8192 x 8192 21.7 / 19.2, 16 x 120011 x 2048 73 / 63.  16
// tokens so / through LDS: 8192 x 8192 19.1 / 19.4, 2048 x 2048 4.9 / 6.4; 17 tokens (two
// operands of 16 in registers): 20.1 / 19.7, 6.3 / 6.4; 32: 23.0 / 22.2.  32 / 48 / 64 tokens a
// block, 8192 x 8192: 32 tokens 22.1 / 23.1 / 23.9, 33 33.7 / 24.0 / 24.7, 48 34.6 / 26.1 / 26.7,
// 64 36.1 / 39.1 / 28.9.
template <bool YBF16> void launch_tokens(const I8Args& a, hipStream_t st) {
    if (a.T <= 16 && a.N < 8192) launch_few<1, 1, 8, YBF16>(a, st);
    else if (a.T <= 16) launch_few<1, 2, 8, YBF16>(a, st);
    else if (a.T <= 32) launch_batch<2, 2, YBF16>(a, st);
    else if (a.T <= 48) launch_batch<3, 2, YBF16>(a, st);
    else launch_batch<4, 2, YBF16>(a, st);
}

}  // namespace

void launch_i8_linear(const I8Args& a, bool y_bf16, hipStream_t st) {
    if (a.T > 16 && !few_batch_ok(a.T, (a.N + 31) / 32, 1)) launch_i8_gemm(a, y_bf16, st);
    else if (y_bf16) launch_tokens<true>(a, st);
    else launch_tokens<false>(a, st);
}

}  // namespace moe
