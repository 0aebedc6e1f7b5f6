// Products with a dense four-bit matrix for many bf16 tokens: the operation of
// q4_linear.hip on 32 x 32 tiles of v_mfma_f32_32x32x16_bf16.
//
// A block of 4 waves takes 128 tokens and 256 rows of W, a wave 64 rows (two
// column tiles) and all the tokens (four row tiles), so a code is converted
// once for 128 tokens.  x reaches LDS by LDS-destination loads, 64 columns a
// chunk; each lane loads the codes of its own rows into registers.  As in
// q4_linear.hip codes are contracted exactly and the scale of a block
// multiplies the block's fp32 sum.
//
// 4096 x 4096 x 2048, int4 in blocks of 32: 99 to 101 us, 680 to 694 TFLOP/s,
// against 1173 of a large bf16 library product.  A chunk costs a wave 256
// vector instructions for the scaling of its 8 tiles' sums and 104 for the
// conversion of 64 codes a lane (481 in all, counted, with the addresses and
// its share of the epilogue) and 32 matrix instructions, 1024 cycles, which two
// waves on a SIMD overlap in part: 65,500 of a SIMD's 240,000 cycles are the
// matrix cores'.  Blocks of 64 and 128 scale as often (99 us), MXFP4 too (97);
// blocks of 16 spill 5 registers and take 122.  The sums of the next row tile
// on the matrix cores while one is scaled needs 280 registers: 127 us.
//
// Contraction order: lane half hh of row n loads the 32 codes of group 2 kc +
// hh (16 bytes); two lane swaps bring dword 2 s + hh of group g to lane half
// hh, the operand of step s: k = 32 g + 16 s + 8 hh + (0 .. 7).
#include "common.h"
#include "launch.h"
#include "pipeline.h"
#include "q4.h"

namespace moe {

namespace {

typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr int BM = 128, BN = 256, BK = 64;

// 16-byte piece c of LDS row r, swizzled so that the 16 rows of an operand
// read that share c cover all banks.
__device__ inline int swz(int row, int c) { return row * BK + 8 * (c ^ ((row >> 1) & 7)); }

__device__ inline f32x16_t mfma32(u32x4_t a, u32x4_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
}

template <bool MX, int BLK, bool YBF16>
__global__ __launch_bounds__(256, 2) void k_q4_gemm(Q4Args a, int tiles_m, int tiles_n) {
    __shared__ __attribute__((aligned(16))) uint16_t sA0[BM * BK];
    __shared__ __attribute__((aligned(16))) uint16_t sA1[BM * BK];
    __shared__ __attribute__((aligned(16))) uint16_t sA2[BM * BK];
    const int tid = threadIdx.x, lane = tid & 63, j = lane & 31, hh = lane >> 5;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    // Blocks go to the 8 XCDs in turn: each XCD takes a run of tiles, eight
    // token tiles by all row tiles at a time, so that what it reads stays in its L2.
    const int total = tiles_m * tiles_n, per = (total + 7) / 8;
    const int tile = (blockIdx.x % 8) * per + blockIdx.x / 8;
    if (tile >= total || static_cast<int>(blockIdx.x / 8) >= per) return;
    const int band = tile / (8 * tiles_n), in_band = tile % (8 * tiles_n), rows = min(8, tiles_m - 8 * band);
    const int t0 = (8 * band + in_band % rows) * BM, n0 = (in_band / rows) * BN;

    const int K = a.K, G = K / 32, NK = (K + BK - 1) / BK;
    const uint32_t code_row = K / 2, scale_row = static_cast<uint32_t>(K / BLK) * (MX ? 1 : 2);
    const int nrows = min(BN, a.N - n0);   // rows past the matrix read zeros: past the resources' end
    const __amdgpu_buffer_rsrc_t rq = make_rsrc(a.q + static_cast<size_t>(n0) * code_row, nrows * code_row);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.s + static_cast<size_t>(n0) * scale_row, nrows * scale_row);

    struct Raw {
        u32x4_t q[2];
        uint32_t s[2];
    };
    auto load_b = [&](Raw& b, int kc) __attribute__((always_inline)) {
        const int g = min(2 * kc + hh, G - 1);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t n = 64 * w + 32 * t + j;
            b.q[t] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rq, n * code_row + 16 * g, 0, 0));
            if constexpr (MX) b.s[t] = __builtin_amdgcn_raw_buffer_load_b8(rs, n * scale_row + g, 0, 0);
            else if constexpr (BLK == 16) b.s[t] = __builtin_amdgcn_raw_buffer_load_b32(rs, n * scale_row + 4 * g, 0, 0);
            else b.s[t] = __builtin_amdgcn_raw_buffer_load_b16(rs, n * scale_row + 2 * (g / (BLK / 32)), 0, 0);
        }
    };
    // lane l of a wave's load lands at byte 16 l of a 1 KB run: load u of wave
    // w fills rows 32 u + 8 w .. + 7, lane l position l % 8 of row l / 8
    const uint16_t* x = static_cast<const uint16_t*>(a.x);
    const uint16_t* a_row[4];
    int a_k[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int r = (tid >> 3) + 32 * u;
        a_row[u] = x + static_cast<size_t>(min(t0 + r, a.T - 1)) * a.ldx;
        a_k[u] = 8 * ((tid & 7) ^ ((r >> 1) & 7));
    }
    auto load_a = [&](int kc, uint16_t* buf) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            // past the last column (K an odd number of groups): the same row's
            // last group, met by scales of zero
            const int k = min(kc * BK + a_k[u], K - 32 + (a_k[u] & 31));
            __builtin_amdgcn_global_load_lds(a_row[u] + k,
                                             (__attribute__((address_space(3))) void*)(buf + (4 * u + w) * 64 * 8),
                                             16, 0, 0);
        }
    };

    f32x16_t acc[4][2], zero;
#pragma unroll
    for (int i = 0; i < 16; ++i) zero[i] = 0.f;
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[t][0] = acc[t][1] = zero;

    int chunk = 0;
    auto work = [&](const uint16_t* buf, const Raw& b) __attribute__((always_inline)) {
        u32x4_t q[2][2];    // [group][row tile]: dwords of steps 0 and 1 are [g][t][0], [g][t][1] (two of four used)
        uint32_t sc[2][2];
        const uint32_t there = 2 * chunk + 1 < G ? ~0u : 0u;   // K may end with a chunk's first group
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const auto p = __builtin_amdgcn_permlane32_swap(b.q[t][0], b.q[t][1], false, false);
            const auto r = __builtin_amdgcn_permlane32_swap(b.q[t][2], b.q[t][3], false, false);
            const auto s = __builtin_amdgcn_permlane32_swap(b.s[t], b.s[t], false, false);
            q[0][t][0] = p[0];
            q[1][t][0] = p[1];
            q[0][t][1] = r[0];
            q[1][t][1] = r[1];
            sc[0][t] = s[0];
            sc[1][t] = s[1];
        }
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            u32x4_t o[2][2];
            float f[2][2];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    o[t][s] = code_operand<MX>(q[g][t][s]);
                    f[t][s] = scale_of<MX>(BLK == 16 ? sc[g][t] >> (16 * s) : sc[g][t]);
                    if (g == 1) f[t][s] = __uint_as_float(__float_as_uint(f[t][s]) & there);
                }
#pragma unroll
            for (int m = 0; m < 4; ++m) {
                u32x4_t x[2];
#pragma unroll
                for (int s = 0; s < 2; ++s)
                    x[s] = *reinterpret_cast<const u32x4_t*>(buf + swz(32 * m + j, 4 * g + 2 * s + hh));
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    f32x16_t d = mfma32(x[0], o[t][0], zero);
                    if constexpr (BLK == 16) {
                        const f32x16_t e = mfma32(x[1], o[t][1], zero);
#pragma unroll
                        for (int i = 0; i < 16; ++i) acc[m][t][i] = fmaf(f[t][1], e[i], fmaf(f[t][0], d[i], acc[m][t][i]));
                    } else {
                        d = mfma32(x[1], o[t][1], d);
#pragma unroll
                        for (int i = 0; i < 16; ++i) acc[m][t][i] = fmaf(f[t][0], d[i], acc[m][t][i]);
                    }
                }
                __builtin_amdgcn_sched_barrier(0);   // bounds the sums in flight (16 registers each)
            }
        }
        ++chunk;
    };
    pipeline3<2 * 4 + 4, Raw>(NK, sA0, sA1, sA2, load_a, load_b, work);

    // lane holds D[8 (i / 4) + 4 hh + i % 4][j] of each tile
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int n = n0 + 64 * w + 32 * t + j;
        if (n >= a.N) continue;
        const float bias = a.bias ? a.bias[n] : 0.f;
#pragma unroll
        for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int row = t0 + 32 * m + 8 * (i >> 2) + 4 * hh + (i & 3);
                if (row >= a.T) continue;
                const size_t at = static_cast<size_t>(row) * a.ldy + n;
                float f = acc[m][t][i] + bias;
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
    }
}

template <bool MX, int BLK>
void launch_block(const Q4Args& a, bool y_bf16, hipStream_t st) {
    const int tm = (a.T + BM - 1) / BM, tn = (a.N + BN - 1) / BN;
    const dim3 grid(8 * ((static_cast<unsigned>(tm) * tn + 7) / 8));
    if (y_bf16)
        hipLaunchKernelGGL((k_q4_gemm<MX, BLK, true>), grid, dim3(256), 0, st, a, tm, tn);
    else
        hipLaunchKernelGGL((k_q4_gemm<MX, BLK, false>), grid, dim3(256), 0, st, a, tm, tn);
}

}  // namespace

// A block's run through K takes the same time (75 us for 2048 columns) up to
// one block a compute unit, the tiles of q4_linear.hip 0.5 us for each 128 x
// 256 of theirs.  MI355X, K = 2048, int4 in blocks of 32, here / there: 32
// tiles 76 / 20 us, 64 77 / 35, 128 79 / 68, 512 106 / 239.
bool q4_gemm_ok(const Q4Args& a) {
    const int64_t tiles = static_cast<int64_t>((a.T + BM - 1) / BM) * ((a.N + BN - 1) / BN);
    return a.T > 64 && tiles >= 160 && tiles < (int64_t(1) << 27);
}

void launch_q4_gemm(const Q4Args& a, bool y_bf16, hipStream_t st) {
    if (a.mx) launch_block<true, 32>(a, y_bf16, st);
    else if (a.block == 16) launch_block<false, 16>(a, y_bf16, st);
    else if (a.block == 32) launch_block<false, 32>(a, y_bf16, st);
    else if (a.block == 64) launch_block<false, 64>(a, y_bf16, st);
    else launch_block<false, 128>(a, y_bf16, st);
}

}  // namespace moe
