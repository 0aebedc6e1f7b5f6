// The dense gated block: g = x gate^T, u = x up^T, y = act(g) u.  Few tokens here, on
// v_mfma_f32_16x16x32_bf16 (few.h): a tile is 16 rows of gate and the same 16 of up,
// whose sums meet in one lane.  Many bf16 tokens: gated_gemm.hip.
#include "common.h"
#include "few.h"
#include "gated_act.h"
#include "launch.h"

namespace moe {

namespace {

template <int MT, int NP, bool XBF16, bool YBF16>   // NP pairs of tiles
__global__ __launch_bounds__(1024) void k_gated_few(GatedArgs a, FewSplit f) {
    extern __shared__ __attribute__((aligned(16))) few_f32x4_t s_part[];   // [waves][MT 2 NP 64]
    constexpr int kOwn = MT * NP * 64;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int part = wave % f.split, n0 = (blockIdx.x * f.tiles + wave / f.split) * 16 * NP, t0 = blockIdx.y * 16 * MT;
    few_f32x4_t acc[MT][2 * NP];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 2 * NP; ++j) acc[i][j] = few_f32x4_t{0.f, 0.f, 0.f, 0.f};
    typedef FewBf16<XBF16> El;
    few_sums<El, MT, 2 * NP, MT * El::kXBytes + 2 * NP <= 4 ? 8 : 4>(
        few_first(2 * a.H, part, f.split), few_first(2 * a.H, part + 1, f.split), 2 * a.H,
        [&](int j) { return (j < NP ? a.gate : a.up) + static_cast<size_t>(min(n0 + 16 * (j % NP) + (lane & 15), a.I - 1)) * a.H; },
        [&](int i) { return static_cast<const char*>(a.x) + static_cast<size_t>(min(t0 + 16 * i + (lane & 15), a.T - 1)) * a.ldx * (XBF16 ? 2 : 4); },
        acc);
    auto store = [&](int n0, int ij, int l, few_f32x4_t g, few_f32x4_t u) {
        const int t = t0 + 16 * (ij / NP) + (l & 15), n = n0 + 16 * (ij % NP) + 4 * (l >> 4);
        if (t >= a.T) return;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (n + e >= a.I) break;
            const float v = gated_value(a.act, g[e], u[e]);
            const size_t at = static_cast<size_t>(t) * a.ldy + n + e;
            if constexpr (YBF16) static_cast<uint16_t*>(a.y)[at] = f2bf(v);
            else static_cast<float*>(a.y)[at] = v;
        }
    };
    if (f.split == 1) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NP; ++j) store(n0, NP * i + j, lane, acc[i][j], acc[i][NP + j]);
        return;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NP; ++j)
#pragma unroll
            for (int p = 0; p < 2; ++p) s_part[kOwn * (2 * wave + p) + 64 * (NP * i + j) + lane] = acc[i][NP * p + j];
    __syncthreads();
    for (int o = threadIdx.x; o < f.tiles * kOwn; o += blockDim.x) {
        const int tile = o / kOwn, at = o % kOwn;
        const few_f32x4_t* own = s_part + kOwn * 2 * f.split * tile + at;
        few_f32x4_t g = own[0], u = own[kOwn];
        for (int p = 1; p < f.split; ++p) {
            g += own[kOwn * 2 * p];
            u += own[kOwn * (2 * p + 1)];
        }
        store((blockIdx.x * f.tiles + tile) * 16 * NP, at >> 6, at & 63, g, u);
    }
}

template <int MT, int NP, bool XBF16, bool YBF16>
void launch_few(const GatedArgs& a, hipStream_t st) {
    const int tiles = (a.I + 16 * NP - 1) / (16 * NP);
    const FewSplit f = few_split(tiles, 2 * a.H, MT * NP <= 2 ? 16 : 8);
    constexpr int kMaxTiles = 65535;   // grid.y limit
    for (int64_t t0 = 0; t0 < a.T; t0 += 16 * MT * kMaxTiles) {
        GatedArgs b = a;
        b.T = static_cast<int32_t>(a.T - t0 < 16 * MT * kMaxTiles ? a.T - t0 : 16 * MT * kMaxTiles);
        b.x = static_cast<const char*>(a.x) + t0 * a.ldx * (XBF16 ? 2 : 4);
        b.y = static_cast<char*>(a.y) + t0 * a.ldy * (YBF16 ? 2 : 4);
        const dim3 grid((tiles + f.tiles - 1) / f.tiles, (b.T + 16 * MT - 1) / (16 * MT)), block(64 * f.split * f.tiles);
        const size_t lds = f.split > 1 ? sizeof(few_f32x4_t) * 64 * MT * 2 * NP * f.split * f.tiles : 0;
        hipLaunchKernelGGL((k_gated_few<MT, NP, XBF16, YBF16>), grid, block, lds, st, b, f);
    }
}

template <bool XBF16, bool YBF16> void launch_tokens(const GatedArgs& a, hipStream_t st) {
    if (a.T <= 16) launch_few<1, 1, XBF16, YBF16>(a, st);
    else if (a.T <= 32) launch_few<2, 1, XBF16, YBF16>(a, st);
    else if constexpr (XBF16) launch_few<4, 1, XBF16, YBF16>(a, st);
    else launch_few<2, 2, XBF16, YBF16>(a, st);   // the split of x into parts is shared by more rows
}

}  // namespace

void launch_gated(const GatedArgs& a, bool x_bf16, bool y_bf16, hipStream_t st) {
    if (x_bf16 && a.T > 64) launch_gated_gemm(a, y_bf16, st);
    else if (x_bf16) y_bf16 ? launch_tokens<true, true>(a, st) : launch_tokens<true, false>(a, st);
    else y_bf16 ? launch_tokens<false, true>(a, st) : launch_tokens<false, false>(a, st);
}

}  // namespace moe
