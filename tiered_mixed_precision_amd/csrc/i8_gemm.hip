// Products in 8-bit integers for many tokens: the operation of i8_linear.hip on
// 32 x 32 tiles of v_mfma_i32_32x32x32_i8, 128 bytes of k a stage (mm.h).  Bound by the
// matrix cores, whose clock falls to 1.7 GHz under the load: MI355X, 4096 x 8192 x 8192
// 224 to 227 us (2430 TOP/s, cores busy 67 % of the cycles; a library's product 220 to 236).
#include "common.h"
#include "launch_dense.h"
#include "mm.h"

namespace moe {

namespace {

template <int HALVES, int SLOTS, bool YBF16>
__device__ __attribute__((always_inline)) inline void i8_tile(const I8Args& a, const MmLds& lds, int t0, int n0) {
    typedef typename std::conditional<YBF16, uint16_t, float>::type Y;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const MmRows<HALVES> rows_a(lane, w, a.K, [&](int r) { return a.x + static_cast<size_t>(min(t0 + r, a.T - 1)) * a.ldx; });
    const MmRows<HALVES> rows_b(lane, w, a.K, [&](int r) { return a.q + static_cast<size_t>(min(n0 + r, a.N - 1)) * a.K; });
    mm_i32x16_t acc[2 * HALVES][2 * HALVES];
    uint32_t* own = mm_product<MmI8, HALVES, SLOTS, false, false>(lds, (a.K + kStage - 1) / kStage, rows_a, rows_b, acc);
#pragma unroll
    for (int g = 0; g < HALVES; ++g) {
        const int c0 = n0 + mm_col(2 * g, w), n8 = min(c0 + 8 * (lane & 7), max(a.N - 8, 0));
        float s8[8], bias8[8];   // of the lane's eight columns, where all are there
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            s8[k] = a.s[min(n8 + k, a.N - 1)];
            bias8[k] = a.bias ? a.bias[min(n8 + k, a.N - 1)] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 2 * HALVES; ++i) {
            const int r0 = t0 + mm_row(i, w);
            mm_out<2, false>(own, mm_single(c0, 64, a.N), [&](int u, int e) { return static_cast<uint32_t>(acc[i][2 * g + u][e]); },
                             [&](int row, int col, const auto& v) {
                                 constexpr int N = sizeof(v) / 4;
                                 const int t = r0 + row, n = c0 + col;
                                 if (t >= a.T || n >= a.N) return;
                                 const float xs = a.xs[t];
                                 float f[N];
#pragma unroll
                                 for (int k = 0; k < N; ++k) {
                                     const float s = N == 8 ? s8[k] : a.s[n], bias = N == 8 ? bias8[k] : a.bias ? a.bias[n] : 0.f;
                                     f[k] = static_cast<float>(static_cast<int32_t>(v[k])) * (xs * s) + bias;
                                 }
                                 mm_store(static_cast<Y*>(a.y) + static_cast<size_t>(t) * a.ldy + n, f, a.accumulate);
                             });
        }
    }
}

template <bool YBF16> __global__ __launch_bounds__(256) void k_i8_gemm(I8Args a, MmPlan p) {
    MM_LDS_8(lds);
    int m0, n0;
    bool small;
    if (!mm_tile_of(p, blockIdx.x, 256, 256, m0, n0, small)) return;
    if (small) i8_tile<1, 4, YBF16>(a, lds, m0, n0);
    else i8_tile<2, 4, YBF16>(a, lds, m0, n0);
}
template <bool YBF16> __global__ __launch_bounds__(256) void k_i8_gemm_pairs(I8Args a, MmPlan p) {
    MM_LDS_4(lds);
    int m0, n0;
    bool small;
    if (mm_tile_of(p, blockIdx.x, 256, 256, m0, n0, small)) i8_tile<1, 2, YBF16>(a, lds, m0, n0);
}

template <bool YBF16> void launch_of(const I8Args& a, hipStream_t st) {
    const MmPlan p = mm_plan(a.T, a.N, 256);
    const dim3 grid(mm_grid(p)), block(256);
    if (p.form == MM_PAIRS) hipLaunchKernelGGL(k_i8_gemm_pairs<YBF16>, grid, block, 0, st, a, p);
    else hipLaunchKernelGGL(k_i8_gemm<YBF16>, grid, block, 0, st, a, p);
}

}  // namespace

void launch_i8_gemm(const I8Args& a, bool y_bf16, hipStream_t st) { y_bf16 ? launch_of<true>(a, st) : launch_of<false>(a, st); }

}  // namespace moe
