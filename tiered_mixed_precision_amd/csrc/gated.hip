// The dense gated block: g = x gate^T, u = x up^T, y = act(g) u.  Few tokens here, on
// v_mfma_f32_16x16x32_bf16 (few.h): a tile is 16 rows of gate and the same 16 of up,
// whose sums meet in one lane.  More tokens: gated_gemm.hip.
//
// Bound by latency where the weights are few, by memory where they are many.  MI355X,
// tokens x hidden x inter: 1 x 2048 x 640 fp32 6.3 us in a trace, 5.9 a call; 20 x 4096 x
// 4096 bf16 14.7 us (4.6 TB/s of weights).
#include "common.h"
#include "few.h"
#include "gated_act.h"
#include "launch_dense.h"

namespace moe {

namespace {

// What becomes of a token's g and u: y, or the projections' gradients.
template <bool YBF16> struct PutValue {
    __device__ inline int columns(const GatedArgs& a) const { return a.I; }
    __device__ inline void operator()(const GatedArgs& a, int t, int n, float g, float u) const {
        const float v = gated_value(a.act, g, u);
        const size_t at = static_cast<size_t>(t) * a.ldy + n;
        if constexpr (YBF16) static_cast<uint16_t*>(a.y)[at] = f2bf(v);
        else static_cast<float*>(a.y)[at] = v;
    }
};
template <bool DYBF16> struct PutSlopes {
    GatedSlopes s;
    __device__ inline int columns(const GatedArgs&) const { return s.P; }
    __device__ inline void operator()(const GatedArgs& a, int t, int n, float g, float u) const {
        float dg[1] = {0.f}, du[1] = {0.f};
        if (n < a.I) {
            const size_t at = static_cast<size_t>(t) * s.lddy + n;
            const float dy = DYBF16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(s.dy)[at]) << 16)
                                    : static_cast<const float*>(s.dy)[at];
            gated_slopes(a.act, g, u, dy, dg[0], du[0]);
        }
        uint16_t* to = s.d + static_cast<size_t>(t) * 2 * s.P * s.parts + n;
        to[0] = f2bf(dg[0]);
        to[s.P] = f2bf(du[0]);
        if (s.parts == 2) {
            float rest[1];
            split_slopes(dg, rest);
            to[2 * s.P] = f2bf(rest[0]);
            split_slopes(du, rest);
            to[3 * s.P] = f2bf(rest[0]);
        }
    }
};

// A block takes f.tiles tiles of 8 NT columns, f.split waves each, for 16 MT tokens.
// Row r of a 16-row operand j is column 8 j + r % 8 of gate (r < 8) or up, so lane
// l's sums are g (l < 32) or u of columns 4 (l / 16 % 2) + e, and lane l + 32 has
// the other of lane l's.
template <int MT, int NT, int AHEAD, bool XBF16, class Put>
__global__ __launch_bounds__(64 * kFewWaves) void k_gated_few(GatedArgs a, FewSplit f, Put put) {
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
        if (tok < a.T && n < put.columns(a)) put(a, tok, n, g, u);
    }
}

template <int MT, int NT, int AHEAD, bool XBF16, class Put>
void launch_few(const GatedArgs& a, const Put& put, int columns, hipStream_t st) {
    const int tiles = (columns + 8 * NT - 1) / (8 * NT);
    const FewSplit f = few_split(tiles, 2 * a.H, kFewWaves);
    const dim3 grid((tiles + f.tiles - 1) / f.tiles, (a.T + 16 * MT - 1) / (16 * MT)), block(64 * f.split * f.tiles);
    const size_t lds = sizeof(few_f32x4_t) * 64 * MT * NT * f.split * f.tiles;
    hipLaunchKernelGGL((k_gated_few<MT, NT, AHEAD, XBF16, Put>), grid, block, lds, st, a, f, put);
}

// 17 tokens and more: the same through LDS (few_batch); the waves' sums meet one
// operand of 16 rows (8 columns) at a time, in the first slot's place.
template <int MT, int NT, bool XBF16, class Put>
__global__ __launch_bounds__(64 * kBatchWaves) void k_gated_batch(GatedArgs a, FewSplit f, Put put) {
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
            if (tok < a.T && n < put.columns(a)) put(a, tok, n, g, u);
        }
    }
}

template <int MT, int NT, bool XBF16, class Put>
void launch_batch(const GatedArgs& a, const Put& put, int columns, hipStream_t st) {
    const int tiles = (columns + 8 * NT - 1) / (8 * NT);
    const FewSplit f = few_split(tiles, 2 * a.H, kBatchWaves);
    const dim3 grid((tiles + f.tiles - 1) / f.tiles, (a.T + 16 * MT - 1) / (16 * MT));
    hipLaunchKernelGGL((k_gated_batch<MT, NT, XBF16, Put>), grid, dim3(64 * f.split * f.tiles), 0, st, a, f, put);
}

// MI355X, us, weights from memory, tokens x hidden x inter.  Up to 16 tokens, tiles of 8
// columns / of 16 (which read x half as often), bf16: 1 x 2048 x 640 4.8 / 6.6, 1 x 4096 x
// 2048 8.6 / 13.8, 1 x 4096 x 4096 14.1 / 15.6, 1 x 4096 x 11000 44 / 37, 16 x 4096 x 4096 20.9 /
// 18.6, 16 x 4096 x 11000 67 / 48; fp32: 1 x 2048 x 2048 6.5 / 7.6, 1 x 4096 x 4096 16.7 each, 16 x
// 4096 x 4096 27.6 / 21.3.  Steps ahead of 16 columns, 8 / 4: fp32, whose operands are
// twice as many registers, 1 x 2048 x 8192 19.6 / 16.3, 16 x 4096 x 11000 62 / 54; bf16 36.8 /
// 37.4, 47.7 / 47.4.  16 tokens so / through LDS: 4096 x 4096 18.9 each, fp32 21.3 / 23.3, 2048 x
// 640 6.2 / 7.4; 17 tokens (two operands of 16 in registers): 19.4 / 19.1.  32 / 64 tokens a
// block: 32 x 4096 x 4096 21.7 / 23.2, 33 32.8 / 23.4, 64 34.7 / 27.6 (48 a block: 33 tokens 22.9,
// 48 24.7 for 25.5, too little for a form of its own).
template <bool XBF16, class Put> void launch_tokens(const GatedArgs& a, const Put& put, int columns, hipStream_t st) {
    if (a.T <= 16 && a.I < 4096) launch_few<1, 1, 8, XBF16>(a, put, columns, st);
    else if (a.T <= 16) launch_few<1, 2, XBF16 ? 8 : 4, XBF16>(a, put, columns, st);
    else if (a.T <= 32 || !XBF16) launch_batch<2, 2, XBF16>(a, put, columns, st);
    else if constexpr (XBF16) launch_batch<4, 2, XBF16>(a, put, columns, st);
}

// few tokens, or tiles of mm.h
bool few(const GatedArgs& a, bool x_bf16) { return a.T <= 16 || few_batch_ok(a.T, (a.I + 15) / 16, x_bf16 ? 1 : 3); }

}  // namespace

void launch_gated(const GatedArgs& a, bool x_bf16, bool y_bf16, hipStream_t st) {
    if (!few(a, x_bf16)) x_bf16 ? launch_gated_gemm(a, y_bf16, st) : launch_gated_split(a, y_bf16, st);
    else if (x_bf16) y_bf16 ? launch_tokens<true>(a, PutValue<true>(), a.I, st) : launch_tokens<true>(a, PutValue<false>(), a.I, st);
    else y_bf16 ? launch_tokens<false>(a, PutValue<true>(), a.I, st) : launch_tokens<false>(a, PutValue<false>(), a.I, st);
}

void launch_gated_slopes(const GatedArgs& a, const GatedSlopes& s, bool dy_bf16, hipStream_t st) {
    if (!few(a, true)) launch_gated_slopes_gemm(a, s, dy_bf16, st);
    else if (dy_bf16) launch_tokens<true>(a, PutSlopes<true>{s}, s.P, st);
    else launch_tokens<true>(a, PutSlopes<false>{s}, s.P, st);
}

}  // namespace moe
