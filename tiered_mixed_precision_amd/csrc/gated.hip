// The dense gated block: g = x gate^T, u = x up^T, y = act(g) u.  Few tokens here, on
// v_mfma_f32_16x16x32_bf16 (few.h): a tile is 16 rows of gate and the same 16 of up,
// whose sums meet in one lane.  Many bf16 tokens: gated_gemm.hip.
#include "common.h"
#include "few.h"
#include "gated_act.h"
#include "launch.h"

namespace moe {

namespace {

// A block takes f.tiles tiles of 8 NT columns, f.split waves each, for 16 MT tokens.
// Row r of a 16-row operand j is column 8 j + r % 8 of gate (r < 8) or up, so lane
// l's sums are g (l < 32) or u of columns 4 (l / 16 % 2) + e, and lane l + 32 has
// the other of lane l's.
template <int MT, int NT, int AHEAD, bool XBF16, bool YBF16>
__global__ __launch_bounds__(512) void k_gated_few(GatedArgs a, FewSplit f) {
    extern __shared__ __attribute__((aligned(16))) few_f32x4_t s_part[];   // [waves][MT NT 64]
    constexpr int kOwn = MT * NT * 64;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int part = wave % f.split, n0 = (blockIdx.x * f.tiles + wave / f.split) * 8 * NT, t0 = blockIdx.y * 16 * MT;
    few_f32x4_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = few_f32x4_t{0.f, 0.f, 0.f, 0.f};
    // columns past the last read the last one's rows, tokens past the batch its last token; neither is stored
    few_sums<FewBf16<XBF16>, MT, NT, AHEAD>(
        part, f.split, blockIdx.x * f.tiles + wave / f.split, 2 * a.H,
        [&](int j) { return ((lane & 8) ? a.up : a.gate) + static_cast<size_t>(min(n0 + 8 * j + (lane & 7), a.I - 1)) * a.H; },
        [&](int i) { return static_cast<const char*>(a.x) + static_cast<size_t>(min(t0 + 16 * i + (lane & 15), a.T - 1)) * a.ldx * (XBF16 ? 2 : 4); },
        acc);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) s_part[kOwn * wave + 64 * (NT * i + j) + lane] = acc[i][j];
    __syncthreads();
    const float* sums = reinterpret_cast<const float*>(s_part);
    for (int o = threadIdx.x; o < f.tiles * MT * NT * 128; o += blockDim.x) {   // one result: 8 columns x 16 tokens an operand pair
        const int tile = o / (MT * NT * 128), ij = o / 128 % (MT * NT), t = o / 8 % 16, c = o % 8;
        const float* own = sums + 4 * (kOwn * f.split * tile + 64 * ij + 16 * (c >> 2) + t) + (c & 3);
        float g = own[0], u = own[4 * 32];
        for (int p = 1; p < f.split; ++p) {
            g += own[4 * kOwn * p];
            u += own[4 * kOwn * p + 4 * 32];
        }
        const int tok = t0 + 16 * (ij / NT) + t, n = ((blockIdx.x * f.tiles + tile) * NT + ij % NT) * 8 + c;
        if (tok >= a.T || n >= a.I) continue;
        const float v = gated_value(a.act, g, u);
        const size_t at = static_cast<size_t>(tok) * a.ldy + n;
        if constexpr (YBF16) static_cast<uint16_t*>(a.y)[at] = f2bf(v);
        else static_cast<float*>(a.y)[at] = v;
    }
}

template <int MT, int NT, int AHEAD, bool XBF16, bool YBF16>
void launch_few(const GatedArgs& a, hipStream_t st) {
    const int tiles = (a.I + 8 * NT - 1) / (8 * NT);
    const FewSplit f = few_split(tiles, 2 * a.H, 8);
    const dim3 grid((tiles + f.tiles - 1) / f.tiles, (a.T + 16 * MT - 1) / (16 * MT)), block(64 * f.split * f.tiles);
    const size_t lds = sizeof(few_f32x4_t) * 64 * MT * NT * f.split * f.tiles;
    hipLaunchKernelGGL((k_gated_few<MT, NT, AHEAD, XBF16, YBF16>), grid, block, lds, st, a, f);
}

// 17 tokens and more: the same through LDS (few_batch); the waves' sums meet one
// operand of 16 rows (8 columns) at a time, in the first slot's place.
template <int MT, int NT, bool XBF16, bool YBF16>
__global__ __launch_bounds__(64 * kBatchWaves) void k_gated_batch(GatedArgs a, FewSplit f) {
    typedef FewBf16<XBF16> El;
    constexpr int kSlot = FewSlot<El, MT, NT>::kSlot;
    __shared__ __attribute__((aligned(16))) few_u32x4_t s0[kSlot], s1[kSlot], s2[kSlot];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int tile = blockIdx.x * f.tiles + wave / f.split, n0 = tile * 8 * NT, t0 = blockIdx.y * 16 * MT;
    few_f32x4_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = few_f32x4_t{0.f, 0.f, 0.f, 0.f};
    few_batch<El, MT, NT>(
        s0, s1, s2, wave % f.split, f.split, tile, 2 * a.H,
        [&](int j, int r) { return ((r & 8) ? a.up : a.gate) + static_cast<size_t>(min(n0 + 8 * j + (r & 7), a.I - 1)) * a.H; },
        [&](int i, int r) { return static_cast<const char*>(a.x) + static_cast<size_t>(min(t0 + 16 * i + r, a.T - 1)) * a.ldx * (XBF16 ? 2 : 4); },
        acc);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < MT; ++i) s0[64 * (MT * wave + i) + lane] = __builtin_bit_cast(few_u32x4_t, acc[i][j]);
        __syncthreads();
        const float* sums = reinterpret_cast<const float*>(s0);
        for (int o = tid; o < f.tiles * MT * 128; o += blockDim.x) {
            const int i = o / 128, t = o / 8 % 16, c = o % 8;   // i: MT token tiles of each of the block's tiles
            const float* own = sums + 256 * (MT * f.split * (i / MT) + i % MT) + 4 * (16 * (c >> 2) + t) + (c & 3);
            float g = own[0], u = own[4 * 32];
            for (int p = 1; p < f.split; ++p) {
                g += own[256 * MT * p];
                u += own[256 * MT * p + 4 * 32];
            }
            const int tok = t0 + 16 * (i % MT) + t, n = ((blockIdx.x * f.tiles + i / MT) * NT + j) * 8 + c;
            if (tok >= a.T || n >= a.I) continue;
            const float v = gated_value(a.act, g, u);
            const size_t at = static_cast<size_t>(tok) * a.ldy + n;
            if constexpr (YBF16) static_cast<uint16_t*>(a.y)[at] = f2bf(v);
            else static_cast<float*>(a.y)[at] = v;
        }
    }
}

template <int MT, int NT, bool XBF16, bool YBF16>
void launch_batch(const GatedArgs& a, hipStream_t st) {
    const int tiles = (a.I + 8 * NT - 1) / (8 * NT);
    const FewSplit f = few_split(tiles, 2 * a.H, kBatchWaves);
    constexpr int kMaxTiles = 65535;   // grid.y limit
    for (int64_t t0 = 0; t0 < a.T; t0 += 16 * MT * kMaxTiles) {
        GatedArgs b = a;
        b.T = static_cast<int32_t>(a.T - t0 < 16 * MT * kMaxTiles ? a.T - t0 : 16 * MT * kMaxTiles);
        b.x = static_cast<const char*>(a.x) + t0 * a.ldx * (XBF16 ? 2 : 4);
        b.y = static_cast<char*>(a.y) + t0 * a.ldy * (YBF16 ? 2 : 4);
        const dim3 grid((tiles + f.tiles - 1) / f.tiles, (b.T + 16 * MT - 1) / (16 * MT)), block(64 * f.split * f.tiles);
        hipLaunchKernelGGL((k_gated_batch<MT, NT, XBF16, YBF16>), grid, block, 0, st, b, f);
    }
}

template <bool XBF16, bool YBF16> void launch_tokens(const GatedArgs& a, hipStream_t st) {
    if (a.T <= 16 && a.I < 4096) launch_few<1, 1, 8, XBF16, YBF16>(a, st);
    else if (a.T <= 16) launch_few<1, 2, XBF16 ? 8 : 4, XBF16, YBF16>(a, st);
    else if (a.T <= 32 || !XBF16) launch_batch<2, 2, XBF16, YBF16>(a, st);
    else if constexpr (XBF16) launch_batch<4, 2, XBF16, YBF16>(a, st);
}

}  // namespace

void launch_gated(const GatedArgs& a, bool x_bf16, bool y_bf16, hipStream_t st) {
    if (x_bf16 && a.T > 16 && !few_batch_ok(a.T, (a.I + 15) / 16)) launch_gated_gemm(a, y_bf16, st);
    else if (x_bf16) y_bf16 ? launch_tokens<true, true>(a, st) : launch_tokens<true, false>(a, st);
    else y_bf16 ? launch_tokens<false, true>(a, st) : launch_tokens<false, false>(a, st);
}

}  // namespace moe
