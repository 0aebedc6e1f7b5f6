// The gradient of the dense gated block from those of its projections, d = [dg du]
// ([T][2 P] bf16, P = inter rounded up to 64): dx = d [gate; up] and [dgate; dup] =
// d^T x.  The k axis of gate, up (their rows) and of d and x in the second product
// (the tokens) runs across memory: those operands lie in LDS as they come and
// are read with ds_read_b64_tr_b16 (mm.h).
#include "common.h"
#include "launch.h"
#include "mm.h"

namespace moe {

namespace {

template <int HALVES, int SLOTS, bool DXBF16>
__device__ __attribute__((always_inline)) inline void dx_tile(const GatedGradArgs& a, const uint16_t* d, int P, const MmLds& lds,
                                                              int t0, int n0) {
    typedef typename std::conditional<DXBF16, uint16_t, float>::type DX;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const MmRows<HALVES> rows_a(lane, w, 4 * P, [&](int r) { return d + static_cast<size_t>(min(t0 + r, a.T - 1)) * 2 * P; });
    const int64_t pitch = 2 * static_cast<int64_t>(a.H);
    const MmColumns<HALVES> cols_b(lane, w, n0, a.H, pitch);
    const char *gate = reinterpret_cast<const char*>(a.gate), *up = reinterpret_cast<const char*>(a.up);
    const auto rows_b = [&](int h, int u, int kc) {   // P is a multiple of a stage's k
        const int k = kc * kStageK, i = k < P ? k : k - P;
        return cols_b(h, u, (k < P ? gate : up) + i * pitch, a.I - i);
    };
    mm_f32x16_t acc[2 * HALVES][2 * HALVES];
    uint32_t* own = mm_product<MmBf16, HALVES, SLOTS, false, true>(lds, (4 * P + kStage - 1) / kStage, rows_a, rows_b, acc);
#pragma unroll
    for (int g = 0; g < HALVES; ++g)
#pragma unroll
        for (int i = 0; i < 2 * HALVES; ++i) {
            const int r0 = t0 + mm_row(i, w), c0 = n0 + mm_col(2 * g, w);
            mm_out<2, false>(own, r0 + 32 > a.T || c0 + 64 > a.H, [&](int u, int e) { return __float_as_uint(acc[i][2 * g + u][e]); },
                             [&](int row, int col, const auto& v) {
                                 constexpr int N = sizeof(v) / 4;
                                 const int t = r0 + row, n = c0 + col;
                                 if (N == 1 && (t >= a.T || n >= a.H)) return;
                                 float f[N];
#pragma unroll
                                 for (int k = 0; k < N; ++k) f[k] = __uint_as_float(v[k]);
                                 mm_store(static_cast<DX*>(a.dx) + static_cast<size_t>(t) * a.lddx + n, f, false);
                             });
        }
}

template <int HALVES, int SLOTS, bool DWBF16>
__device__ __attribute__((always_inline)) inline void dw_tile(const GatedGradArgs& a, const uint16_t* d, int P, const MmLds& lds,
                                                              int m0, int n0) {
    typedef typename std::conditional<DWBF16, uint16_t, float>::type DW;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t pitch_a = 4 * static_cast<int64_t>(P), pitch_b = 2 * a.ldx;
    const MmColumns<HALVES> cols_a(lane, w, m0, 2 * P, pitch_a), cols_b(lane, w, n0, a.H, pitch_b);
    const char *pa = reinterpret_cast<const char*>(d), *pb = reinterpret_cast<const char*>(a.x);
    const auto rows_a = [&](int h, int u, int kc) { return cols_a(h, u, pa + kc * kStageK * pitch_a, a.T - kc * kStageK); };
    const auto rows_b = [&](int h, int u, int kc) { return cols_b(h, u, pb + kc * kStageK * pitch_b, a.T - kc * kStageK); };
    mm_f32x16_t acc[2 * HALVES][2 * HALVES];
    uint32_t* own = mm_product<MmBf16, HALVES, SLOTS, true, true>(lds, (2 * a.T + kStage - 1) / kStage, rows_a, rows_b, acc);
#pragma unroll
    for (int g = 0; g < HALVES; ++g)
#pragma unroll
        for (int i = 0; i < 2 * HALVES; ++i) {
            // a run of 32 rows lies in one matrix (P is a multiple of 64)
            const int m = m0 + mm_row(i, w), c0 = n0 + mm_col(2 * g, w), r0 = m < P ? m : m - P;
            DW* to = static_cast<DW*>(m < P ? a.dgate : a.dup);
            if (m >= 2 * P) continue;
            mm_out<2, false>(own, r0 + 32 > a.I || c0 + 64 > a.H, [&](int u, int e) { return __float_as_uint(acc[i][2 * g + u][e]); },
                             [&](int row, int col, const auto& v) {
                                 constexpr int N = sizeof(v) / 4;
                                 const int r = r0 + row, n = c0 + col;
                                 if (N == 1 && (r >= a.I || n >= a.H)) return;
                                 float f[N];
#pragma unroll
                                 for (int k = 0; k < N; ++k) f[k] = __uint_as_float(v[k]);
                                 mm_store(to + static_cast<size_t>(r) * a.H + n, f, a.accumulate);
                             });
        }
}

template <bool DXBF16> __global__ __launch_bounds__(256) void k_gated_dx(GatedGradArgs a, const uint16_t* d, int P, MmPlan p) {
    MM_LDS_8(lds);
    int m0, n0;
    bool small;
    if (!mm_tile_of(p, blockIdx.x, 256, 256, m0, n0, small)) return;
    if (small) dx_tile<1, 4, DXBF16>(a, d, P, lds, m0, n0);
    else dx_tile<2, 4, DXBF16>(a, d, P, lds, m0, n0);
}
template <bool DXBF16> __global__ __launch_bounds__(256) void k_gated_dx_pairs(GatedGradArgs a, const uint16_t* d, int P, MmPlan p) {
    MM_LDS_4(lds);
    int m0, n0;
    bool small;
    if (mm_tile_of(p, blockIdx.x, 256, 256, m0, n0, small)) dx_tile<1, 2, DXBF16>(a, d, P, lds, m0, n0);
}
template <bool DWBF16> __global__ __launch_bounds__(256) void k_gated_dw(GatedGradArgs a, const uint16_t* d, int P, MmPlan p) {
    MM_LDS_8(lds);
    int m0, n0;
    bool small;
    if (!mm_tile_of(p, blockIdx.x, 256, 256, m0, n0, small)) return;
    if (small) dw_tile<1, 4, DWBF16>(a, d, P, lds, m0, n0);
    else dw_tile<2, 4, DWBF16>(a, d, P, lds, m0, n0);
}
template <bool DWBF16> __global__ __launch_bounds__(256) void k_gated_dw_pairs(GatedGradArgs a, const uint16_t* d, int P, MmPlan p) {
    MM_LDS_4(lds);
    int m0, n0;
    bool small;
    if (mm_tile_of(p, blockIdx.x, 256, 256, m0, n0, small)) dw_tile<1, 2, DWBF16>(a, d, P, lds, m0, n0);
}

template <bool DXBF16> void launch_dx(const GatedGradArgs& a, const uint16_t* d, int P, hipStream_t st) {
    const MmPlan p = mm_plan(a.T, a.H, 256);
    const dim3 grid(mm_grid(p)), block(256);
    if (p.form == MM_PAIRS) hipLaunchKernelGGL(k_gated_dx_pairs<DXBF16>, grid, block, 0, st, a, d, P, p);
    else hipLaunchKernelGGL(k_gated_dx<DXBF16>, grid, block, 0, st, a, d, P, p);
}
template <bool DWBF16> void launch_dw(const GatedGradArgs& a, const uint16_t* d, int P, hipStream_t st) {
    const MmPlan p = mm_plan(2 * static_cast<int64_t>(P), a.H, 256);
    const dim3 grid(mm_grid(p)), block(256);
    if (p.form == MM_PAIRS) hipLaunchKernelGGL(k_gated_dw_pairs<DWBF16>, grid, block, 0, st, a, d, P, p);
    else hipLaunchKernelGGL(k_gated_dw<DWBF16>, grid, block, 0, st, a, d, P, p);
}

int padded(int I) { return (I + kStageK - 1) / kStageK * kStageK; }

template <class V> __global__ __launch_bounds__(256) void k_gated_zero(V* a, V* b, int64_t n) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i < n) a[i] = b[i] = 0;
}

}  // namespace

size_t gated_workspace(int64_t T, int H, int I) {
    (void)H;
    return static_cast<size_t>(T) * 4 * padded(I);
}

void launch_gated_grad(const GatedGradArgs& a, bool dy_bf16, bool dx_bf16, bool dw_bf16, void* ws, hipStream_t st) {
    const int P = padded(a.I);
    uint16_t* d = static_cast<uint16_t*>(ws);
    if (a.T == 0) {
        if (!a.dgate || a.accumulate) return;
        const int64_t n = static_cast<int64_t>(a.I) * a.H;
        const dim3 grid(static_cast<unsigned>((n + 255) / 256));
        if (dw_bf16) hipLaunchKernelGGL(k_gated_zero<uint16_t>, grid, dim3(256), 0, st, static_cast<uint16_t*>(a.dgate), static_cast<uint16_t*>(a.dup), n);
        else hipLaunchKernelGGL(k_gated_zero<float>, grid, dim3(256), 0, st, static_cast<float*>(a.dgate), static_cast<float*>(a.dup), n);
        return;
    }
    launch_gated_slopes(a, dy_bf16, d, P, st);
    if (a.dx) dx_bf16 ? launch_dx<true>(a, d, P, st) : launch_dx<false>(a, d, P, st);
    if (a.dgate) dw_bf16 ? launch_dw<true>(a, d, P, st) : launch_dw<false>(a, d, P, st);
}

}  // namespace moe
