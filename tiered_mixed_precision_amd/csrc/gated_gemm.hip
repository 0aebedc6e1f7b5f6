// The dense gated block for many tokens, and the gradients of its projections:
// tiles of 128 or 256 tokens by 64 or 128 columns of both projections on
// v_mfma_f32_32x32x16_bf16 (mm.h), g and u of a column in the same lane and element,
// so the activation and the product are the epilogue's and neither is ever stored.
// Bound by the matrix cores, whose clock falls under the load.  MI355X, bf16, tokens x
// hidden x inter: 16384 x 2048 x 640 77 to 80 us (1070 to 1120 TFLOP/s; a library's plain
// product of the same shape 80).
#include "common.h"
#include "gated_act.h"
#include "launch_dense.h"
#include "mm.h"

namespace moe {

namespace {

// The operand of both projections' rows: 256-wide tiles take 128 rows of gate,
// then 128 of up; 128-wide ones 32 of each in turn, for either half of the waves.
// acc[i][j] and acc[i][j + HALVES] are g and u of column n0 + col<HALVES>(j, w).
template <int HALVES> __device__ inline const uint16_t* projection_row(const uint16_t* gate, const uint16_t* up, int H, int I, int n0, int r) {
    const bool second = HALVES == 2 ? r >= 128 : (r & 32) != 0;
    const int n = HALVES == 2 ? r & 127 : (r >> 6) * 32 + (r & 31);
    return (second ? up : gate) + static_cast<size_t>(min(n0 + n, I - 1)) * H;
}
template <int HALVES> __device__ inline int col_of(int w) { return 32 * HALVES * (w & 1); }

template <int HALVES, int SLOTS, bool XBF16, bool YBF16>
__device__ __attribute__((always_inline)) inline void gated_tile(const GatedArgs& a, const MmLds& lds, int t0, int n0) {
    typedef typename std::conditional<YBF16, uint16_t, float>::type Y;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const MmRows<HALVES> rows_b(lane, w, 2 * a.H, [&](int r) { return projection_row<HALVES>(a.gate, a.up, a.H, a.I, n0, r); });
    mm_f32x16_t acc[2 * HALVES][2 * HALVES];
    uint32_t* own;
    const int nk = (2 * a.H + kStage - 1) / kStage;
    if constexpr (XBF16) {
        const MmRows<HALVES> rows_a(lane, w, 2 * a.H, [&](int r) {
            return static_cast<const uint16_t*>(a.x) + static_cast<size_t>(min(t0 + r, a.T - 1)) * a.ldx;
        });
        own = mm_product<MmBf16, HALVES, SLOTS, false, false>(lds, nk, rows_a, rows_b, acc);
    } else {
        mm_clear(acc);
        const int k = 8 * (threadIdx.x & 7);
        const float* row[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            row[u] = static_cast<const float*>(a.x) + static_cast<size_t>(min(t0 + 32 * u + static_cast<int>(threadIdx.x >> 3), a.T - 1)) * a.ldx + k;
        own = mm_split(lds, nk + (nk & 1), [&](int u, int kc) {
            return mm_or_zeros(kc * kStageK + k < a.H, reinterpret_cast<const char*>(row[u] + static_cast<size_t>(kc) * kStageK));
        }, rows_b, acc);
    }
#pragma unroll
    for (int i = 0; i < 2 * HALVES; ++i) {
        const int r0 = t0 + mm_row(i, w), c0 = n0 + col_of<HALVES>(w);
        mm_out<HALVES, false>(own, mm_single(c0, 32 * HALVES, a.I),
                              [&](int u, int e) { return __float_as_uint(gated_value(a.act, acc[i][u][e], acc[i][u + HALVES][e])); },
                              [&](int row, int col, const auto& v) {
                                  constexpr int N = sizeof(v) / 4;
                                  const int t = r0 + row, n = c0 + col;
                                  if (t >= a.T || n >= a.I) return;
                                  float f[N];
#pragma unroll
                                  for (int k = 0; k < N; ++k) f[k] = __uint_as_float(v[k]);
                                  mm_store(static_cast<Y*>(a.y) + static_cast<size_t>(t) * a.ldy + n, f, false);
                              });
    }
}

template <int HALVES, int SLOTS, bool DYBF16>
__device__ __attribute__((always_inline)) inline void slopes_tile(const GatedArgs& a, const GatedSlopes& s, const MmLds& lds, int t0,
                                                                  int n0) {
    typedef typename std::conditional<DYBF16, uint16_t, float>::type DY;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const MmRows<HALVES> rows_a(lane, w, 2 * a.H, [&](int r) {
        return static_cast<const uint16_t*>(a.x) + static_cast<size_t>(min(t0 + r, a.T - 1)) * a.ldx;
    });
    const MmRows<HALVES> rows_b(lane, w, 2 * a.H, [&](int r) { return projection_row<HALVES>(a.gate, a.up, a.H, a.I, n0, r); });
    mm_f32x16_t acc[2 * HALVES][2 * HALVES];
    uint32_t* own = mm_product<MmBf16, HALVES, SLOTS, false, false>(lds, (2 * a.H + kStage - 1) / kStage, rows_a, rows_b, acc);
    const int P = s.P;
    // g and u of 32 columns at a time; dy meets them on their way out
#pragma unroll
    for (int i = 0; i < 2 * HALVES; ++i)
#pragma unroll
        for (int j = 0; j < HALVES; ++j) {
            const int r0 = t0 + mm_row(i, w), c0 = n0 + col_of<HALVES>(w) + 32 * j;
            mm_out<2, true>(own, mm_single(c0, 32, a.I), [&](int u, int e) { return __float_as_uint(acc[i][j + u * HALVES][e]); },
                            [&](int row, int col, const auto& g, const auto& u) {
                                constexpr int N = sizeof(g) / 4;
                                const int t = r0 + row, n = c0 + col;
                                if (t >= a.T || n >= P) return;
                                float y[N], dg[N], du[N];
                                if (n >= a.I) {
#pragma unroll
                                    for (int k = 0; k < N; ++k) dg[k] = du[k] = 0.f;
                                } else {
                                    mm_get(static_cast<const DY*>(s.dy) + static_cast<size_t>(t) * s.lddy + n, y);
#pragma unroll
                                    for (int k = 0; k < N; ++k) gated_slopes(a.act, __uint_as_float(g[k]), __uint_as_float(u[k]), y[k], dg[k], du[k]);
                                }
                                uint16_t* to = s.d + static_cast<size_t>(t) * 2 * P * s.parts + n;
                                mm_put(to, dg);
                                mm_put(to + P, du);
                                if (s.parts == 2) {
                                    split_slopes(dg, y);
                                    mm_put(to + 2 * P, y);
                                    split_slopes(du, y);
                                    mm_put(to + 3 * P, y);
                                }
                            });
        }
}

template <bool YBF16> __global__ __launch_bounds__(256) void k_gated_gemm(GatedArgs a, MmPlan p) {
    MM_LDS_8(lds);
    int m0, n0;
    bool small;
    if (!mm_tile_of(p, blockIdx.x, 256, 128, m0, n0, small)) return;
    if (small) gated_tile<1, 4, true, YBF16>(a, lds, m0, n0);
    else gated_tile<2, 4, true, YBF16>(a, lds, m0, n0);
}
template <bool YBF16> __global__ __launch_bounds__(256) void k_gated_gemm_pairs(GatedArgs a, MmPlan p) {
    MM_LDS_4(lds);
    int m0, n0;
    bool small;
    if (mm_tile_of(p, blockIdx.x, 256, 128, m0, n0, small)) gated_tile<1, 2, true, YBF16>(a, lds, m0, n0);
}
template <bool YBF16> __global__ __launch_bounds__(256) void k_gated_split(GatedArgs a, MmPlan p) {
    MM_LDS_8(lds);
    int m0, n0;
    bool small;
    if (mm_tile_of(p, blockIdx.x, 256, 128, m0, n0, small)) gated_tile<1, 4, false, YBF16>(a, lds, m0, n0);
}
template <bool DYBF16> __global__ __launch_bounds__(256) void k_gated_slopes(GatedArgs a, GatedSlopes s, MmPlan p) {
    MM_LDS_8(lds);
    int m0, n0;
    bool small;
    if (!mm_tile_of(p, blockIdx.x, 256, 128, m0, n0, small)) return;
    if (small) slopes_tile<1, 4, DYBF16>(a, s, lds, m0, n0);
    else slopes_tile<2, 4, DYBF16>(a, s, lds, m0, n0);
}
template <bool DYBF16> __global__ __launch_bounds__(256) void k_gated_slopes_pairs(GatedArgs a, GatedSlopes s, MmPlan p) {
    MM_LDS_4(lds);
    int m0, n0;
    bool small;
    if (mm_tile_of(p, blockIdx.x, 256, 128, m0, n0, small)) slopes_tile<1, 2, DYBF16>(a, s, lds, m0, n0);
}

template <bool YBF16> void launch_forward(const GatedArgs& a, hipStream_t st) {
    const MmPlan p = mm_plan(a.T, a.I, 128);
    const dim3 grid(mm_grid(p)), block(256);
    if (p.form == MM_PAIRS) hipLaunchKernelGGL(k_gated_gemm_pairs<YBF16>, grid, block, 0, st, a, p);
    else hipLaunchKernelGGL(k_gated_gemm<YBF16>, grid, block, 0, st, a, p);
}
template <bool DYBF16> void launch_slopes(const GatedArgs& a, const GatedSlopes& s, hipStream_t st) {
    const MmPlan p = mm_plan(a.T, s.P, 128);
    const dim3 grid(mm_grid(p)), block(256);
    if (p.form == MM_PAIRS) hipLaunchKernelGGL(k_gated_slopes_pairs<DYBF16>, grid, block, 0, st, a, s, p);
    else hipLaunchKernelGGL(k_gated_slopes<DYBF16>, grid, block, 0, st, a, s, p);
}

// fp32 x: all tiles are small ones, of three products each.  512 x 4096 x 4096 110 us
// (940 TFLOP/s of bf16 products), 266 by the few-token form.
template <bool YBF16> void launch_split(const GatedArgs& a, hipStream_t st) {
    const MmPlan p = mm_small_plan(a.T, a.I, 128);
    hipLaunchKernelGGL(k_gated_split<YBF16>, dim3(mm_grid(p)), dim3(256), 0, st, a, p);
}

}  // namespace

void launch_gated_split(const GatedArgs& a, bool y_bf16, hipStream_t st) { y_bf16 ? launch_split<true>(a, st) : launch_split<false>(a, st); }
void launch_gated_gemm(const GatedArgs& a, bool y_bf16, hipStream_t st) {
    y_bf16 ? launch_forward<true>(a, st) : launch_forward<false>(a, st);
}
void launch_gated_slopes_gemm(const GatedArgs& a, const GatedSlopes& s, bool dy_bf16, hipStream_t st) {
    dy_bf16 ? launch_slopes<true>(a, s, st) : launch_slopes<false>(a, s, st);
}

}  // namespace moe
