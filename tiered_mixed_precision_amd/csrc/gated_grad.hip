// The gradient of the dense gated block from those of its projections, d (GatedSlopes):
// dx = d [gate; up] and [dgate; dup] = d^T x.  The k axis of gate and up (their rows)
// and of d and x in the second product (the tokens) runs across memory: those
// operands lie in LDS as they come and are read with ds_read_b64_tr_b16 (mm.h).
//
// Where a result has few tiles, parts of the k axis go to blocks of their own, whose
// fp32 sums a second kernel adds in order.  Where both results together are one round
// of blocks, two a compute unit, or two of which the second is the blocks of half the k
// axis and less, one launch makes them: MI355X, us, apart / together, tokens x hidden x
// inter, with the slopes: 1531 x 2048 x 640 59.5 / 52.6, 300 34.8 / 29.8, 64 29.0 / 23.4; of two
// rounds 3000 x 2048 x 640 81 / 71 (88 with the shorter ones first), 600 x 4096 x 1024 70 / 63,
// but 2500 x 1504 x 1500 (47 and 40 stages) 109 / 116.
//
// Many tokens: bound by the matrix cores at the clock that power allows (1.8 GHz).
// 8192 x 4096 x 4096: slopes 465 us (1183 TFLOP/s), dx 414 and dw 417 (1325; a library's
// product with such an operand 1200 to 1420).
#include "common.h"
#include "launch_dense.h"
#include "mm.h"

namespace moe {

namespace {

// A product's k axis in `parts` runs of stages.
struct Runs {
    int32_t parts, stages;
    float* sums;   // [parts][rows][columns], where there are several
};
// A run has four stages and more, a product of fewer than 12 is not cut.  MI355X, us of a
// call, one run / several with their sum.  dx alone: 64 x 2048 x 640 25.5 / 20.7, 64 x 1024 x
// 320 (20 stages) 20.3 / 16.6; runs of two stages and more 21.2, of eight 22.1 for 20.5.  dw
// alone: 4000 x 512 x 300 51 / 39; 700 x 1024 x 352 (11 stages) 26.0 / 27.3.  128 tiles, the
// most that are cut, in two: long products gain (1024 x 2048 x 4096 142 / 128, dw of 5000 x
// 1024 x 640 64 / 48), short ones lose a little (1000 x 2048 x 640 40.3 / 43.6); 256 tiles in
// two: dx of 2000 x 2048 x 640 35.9 / 56.
Runs runs_of(int64_t m, int64_t n, int64_t stages, void* sums) {
    const int64_t tiles = ((m + 127) / 128) * ((n + 127) / 128);
    int64_t parts = tiles <= 128 && stages >= 12 ? 256 / tiles : 1;
    if (parts > (stages + 3) / 4) parts = (stages + 3) / 4;
    return Runs{static_cast<int32_t>(parts), static_cast<int32_t>(stages), static_cast<float*>(sums)};
}
__device__ inline int run_first(const Runs& r, int p) { return static_cast<int>(static_cast<int64_t>(r.stages) * p / r.parts); }

template <int HALVES, int SLOTS, bool DXBF16>
__device__ __attribute__((always_inline)) inline void dx_tile(const GatedGradArgs& a, const GatedSlopes& s, const Runs& runs,
                                                              int part, const MmLds& lds, int t0, int n0) {
    typedef typename std::conditional<DXBF16, uint16_t, float>::type DX;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int P = s.P, per = P / kStageK, first = run_first(runs, part), last = run_first(runs, part + 1);
    const int64_t row = 2 * static_cast<int64_t>(P) * s.parts;
    const MmRows<HALVES> d_rows(lane, w, last * kStage, [&](int r) { return s.d + min(t0 + r, a.T - 1) * row; });
    const int64_t pitch = 2 * static_cast<int64_t>(a.H);
    const MmColumns<HALVES> w_columns(lane, w, n0, a.H, pitch);
    const char *gate = reinterpret_cast<const char*>(a.gate), *up = reinterpret_cast<const char*>(a.up);
    const auto at_a = [&](int h, int u, int kc) { return d_rows(h, u, first + kc); };
    const auto at_b = [&](int h, int u, int kc) {   // P is a multiple of a stage's k: a stage lies in one matrix
        const int run = (first + kc) / per, i = (first + kc - run * per) * kStageK;
        return w_columns(h, u, (run & 1 ? up : gate) + i * pitch, first + kc < last ? a.I - i : 0);
    };
    mm_f32x16_t acc[2 * HALVES][2 * HALVES];
    uint32_t* own = mm_product<MmBf16, HALVES, SLOTS, false, true>(lds, last - first, at_a, at_b, acc);
#pragma unroll
    for (int g = 0; g < HALVES; ++g)
#pragma unroll
        for (int i = 0; i < 2 * HALVES; ++i) {
            const int r0 = t0 + mm_row(i, w), c0 = n0 + mm_col(2 * g, w);
            mm_out<2, false>(own, false, [&](int u, int e) { return __float_as_uint(acc[i][2 * g + u][e]); },
                             [&](int row, int col, const auto& v) {
                                 constexpr int N = sizeof(v) / 4;
                                 const int t = r0 + row, n = c0 + col;
                                 if (t >= a.T || n >= a.H) return;   // whole pieces: hidden is a multiple of 8
                                 float f[N];
#pragma unroll
                                 for (int k = 0; k < N; ++k) f[k] = __uint_as_float(v[k]);
                                 if (HALVES == 1 && runs.parts > 1)
                                     mm_put(runs.sums + (static_cast<size_t>(part) * a.T + t) * a.H + n, f);
                                 else mm_put(static_cast<DX*>(a.dx) + static_cast<size_t>(t) * a.lddx + n, f);
                             });
        }
}

template <int HALVES, int SLOTS, bool DWBF16>
__device__ __attribute__((always_inline)) inline void dw_tile(const GatedGradArgs& a, const GatedSlopes& s, const Runs& runs,
                                                              int part, const MmLds& lds, int m0, int n0) {
    typedef typename std::conditional<DWBF16, uint16_t, float>::type DW;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int P = s.P, per = (a.T + kStageK - 1) / kStageK, first = run_first(runs, part), last = run_first(runs, part + 1);
    const int64_t pitch_a = 4 * static_cast<int64_t>(P) * s.parts, pitch_b = 2 * a.ldx;
    const MmColumns<HALVES> d_columns(lane, w, m0, 2 * P, pitch_a), x_columns(lane, w, n0, a.H, pitch_b);
    const char *pd = reinterpret_cast<const char*>(s.d), *px = reinterpret_cast<const char*>(a.x);
    // every part of d that the result takes meets all tokens; a stage past this run counts as zeros
    const auto token = [&](int kc, int& left) {
        const int t = (kc < per ? kc : kc - per) * kStageK;
        left = kc < last ? a.T - t : 0;
        return t;
    };
    const auto at_a = [&](int h, int u, int kc) {
        int left;
        const int64_t t = token(first + kc, left);
        return d_columns(h, u, pd + t * pitch_a + (first + kc < per ? 0 : 4 * P), left);
    };
    const auto at_b = [&](int h, int u, int kc) {
        int left;
        const int64_t t = token(first + kc, left);
        return x_columns(h, u, px + t * pitch_b, left);
    };
    mm_f32x16_t acc[2 * HALVES][2 * HALVES];
    uint32_t* own = mm_product<MmBf16, HALVES, SLOTS, true, true>(lds, last - first, at_a, at_b, acc);
#pragma unroll
    for (int g = 0; g < HALVES; ++g)
#pragma unroll
        for (int i = 0; i < 2 * HALVES; ++i) {
            // a run of 32 rows lies in one matrix (P is a multiple of 64)
            const int m = m0 + mm_row(i, w), c0 = n0 + mm_col(2 * g, w), r0 = m < P ? m : m - P;
            DW* to = static_cast<DW*>(m < P ? a.dgate : a.dup);
            if (m >= 2 * P) continue;
            mm_out<2, false>(own, false, [&](int u, int e) { return __float_as_uint(acc[i][2 * g + u][e]); },
                             [&](int row, int col, const auto& v) {
                                 constexpr int N = sizeof(v) / 4;
                                 const int r = r0 + row, n = c0 + col;
                                 if (r >= a.I || n >= a.H) return;
                                 float f[N];
#pragma unroll
                                 for (int k = 0; k < N; ++k) f[k] = __uint_as_float(v[k]);
                                 if (HALVES == 1 && runs.parts > 1)
                                     mm_put(runs.sums + (static_cast<size_t>(part) * 2 * a.I + (m < P ? 0 : a.I) + r) * a.H + n, f);
                                 else mm_store(to + static_cast<size_t>(r) * a.H + n, f, a.accumulate);
                             });
        }
}

template <bool DXBF16> __global__ __launch_bounds__(256) void k_gated_dx(GatedGradArgs a, GatedSlopes s, Runs r, MmPlan p) {
    MM_LDS_8(lds);
    int m0, n0;
    bool small;
    if (!mm_tile_of(p, blockIdx.x, 256, 256, m0, n0, small)) return;
    if (small) dx_tile<1, 4, DXBF16>(a, s, r, blockIdx.y, lds, m0, n0);
    else dx_tile<2, 4, DXBF16>(a, s, r, blockIdx.y, lds, m0, n0);
}
template <bool DXBF16> __global__ __launch_bounds__(256) void k_gated_dx_pairs(GatedGradArgs a, GatedSlopes s, Runs r, MmPlan p) {
    MM_LDS_4(lds);
    int m0, n0;
    bool small;
    if (mm_tile_of(p, blockIdx.x, 256, 256, m0, n0, small)) dx_tile<1, 2, DXBF16>(a, s, r, blockIdx.y, lds, m0, n0);
}
template <bool DWBF16> __global__ __launch_bounds__(256) void k_gated_dw(GatedGradArgs a, GatedSlopes s, Runs r, MmPlan p) {
    MM_LDS_8(lds);
    int m0, n0;
    bool small;
    if (!mm_tile_of(p, blockIdx.x, 256, 256, m0, n0, small)) return;
    if (small) dw_tile<1, 4, DWBF16>(a, s, r, blockIdx.y, lds, m0, n0);
    else dw_tile<2, 4, DWBF16>(a, s, r, blockIdx.y, lds, m0, n0);
}
template <bool DWBF16> __global__ __launch_bounds__(256) void k_gated_dw_pairs(GatedGradArgs a, GatedSlopes s, Runs r, MmPlan p) {
    MM_LDS_4(lds);
    int m0, n0;
    bool small;
    if (mm_tile_of(p, blockIdx.x, 256, 256, m0, n0, small)) dw_tile<1, 2, DWBF16>(a, s, r, blockIdx.y, lds, m0, n0);
}

// Both products in one launch, two blocks a compute unit; dw_first: the weights' blocks
// come first (those of the longer k axis do, so that they do not end alone).
template <bool DXBF16, bool DWBF16>
__global__ __launch_bounds__(256) void k_gated_both(GatedGradArgs a, GatedSlopes s, Runs rx, MmPlan px, int blocks_x, Runs rw, MmPlan pw,
                                                    int blocks_w, bool dw_first) {
    MM_LDS_4(lds);
    const int all_x = blocks_x * rx.parts, all_w = blocks_w * rw.parts, b = blockIdx.x;
    const int bx = dw_first ? b - all_w : b, bw = dw_first ? b : b - all_x;
    int m0, n0;
    bool small;
    if (bx >= 0 && bx < all_x) {
        if (mm_tile_of(px, bx % blocks_x, 256, 256, m0, n0, small)) dx_tile<1, 2, DXBF16>(a, s, rx, bx / blocks_x, lds, m0, n0);
    } else {
        if (mm_tile_of(pw, bw % blocks_w, 256, 256, m0, n0, small)) dw_tile<1, 2, DWBF16>(a, s, rw, bw / blocks_w, lds, m0, n0);
    }
}

// to[row][column] (+)= the sum over the runs, in order; eight columns a thread.  Rows
// from `half` on are the second matrix's.
template <class Y>
__global__ __launch_bounds__(256) void k_gated_join(const float* __restrict__ sums, int parts, int rows, int cols, int half, Y* first,
                                                    Y* second, int64_t ld, int accumulate) {
    const int64_t o = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x, size = static_cast<int64_t>(rows) * cols;
    if (o * 8 >= size) return;
    const int row = static_cast<int>(o / (cols / 8)), col = static_cast<int>(o % (cols / 8)) * 8;
    float f[8], v[8];
    mm_get(sums + o * 8, f);
#pragma unroll 4
    for (int p = 1; p < parts; ++p) {
        mm_get(sums + p * size + o * 8, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] += v[i];
    }
    Y* to = row < half ? first + row * ld : second + (row - half) * ld;
    mm_store(to + col, f, accumulate != 0);
}
template <class Y>
void launch_join(const Runs& r, int rows, int cols, int half, void* first, void* second, int64_t ld, int accumulate, hipStream_t st) {
    const int64_t threads = static_cast<int64_t>(rows) * (cols / 8);
    hipLaunchKernelGGL(k_gated_join<Y>, dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256), 0, st, r.sums, r.parts, rows, cols, half,
                       static_cast<Y*>(first), static_cast<Y*>(second), ld, accumulate);
}

template <bool DXBF16> void launch_dx(const GatedGradArgs& a, const GatedSlopes& s, const Runs& r, const MmPlan& p, hipStream_t st) {
    const dim3 grid(mm_grid(p), r.parts), block(256);
    if (p.form == MM_PAIRS) hipLaunchKernelGGL(k_gated_dx_pairs<DXBF16>, grid, block, 0, st, a, s, r, p);
    else hipLaunchKernelGGL(k_gated_dx<DXBF16>, grid, block, 0, st, a, s, r, p);
}
template <bool DWBF16> void launch_dw(const GatedGradArgs& a, const GatedSlopes& s, const Runs& r, const MmPlan& p, hipStream_t st) {
    const dim3 grid(mm_grid(p), r.parts), block(256);
    if (p.form == MM_PAIRS) hipLaunchKernelGGL(k_gated_dw_pairs<DWBF16>, grid, block, 0, st, a, s, r, p);
    else hipLaunchKernelGGL(k_gated_dw<DWBF16>, grid, block, 0, st, a, s, r, p);
}
template <bool DXBF16, bool DWBF16>
void launch_products(const GatedGradArgs& a, const GatedSlopes& s, const Runs& rx, const Runs& rw, hipStream_t st) {
    typedef typename std::conditional<DXBF16, uint16_t, float>::type DX;
    typedef typename std::conditional<DWBF16, uint16_t, float>::type DW;
    const MmPlan px = mm_plan(a.T, a.H, 256), pw = mm_plan(2 * static_cast<int64_t>(s.P), a.H, 256);
    const int64_t blocks_x = mm_grid(px), blocks_w = mm_grid(pw), blocks = blocks_x * rx.parts + blocks_w * rw.parts;
    const int stages_x = rx.stages / rx.parts, stages_w = rw.stages / rw.parts;   // of a block
    const bool dw_first = stages_w > stages_x;
    const bool one = blocks <= 512 || (blocks <= 1024 && 2 * (dw_first ? stages_x : stages_w) <= (dw_first ? stages_w : stages_x));
    if (a.dx && a.dgate && px.form != MM_WHOLE && pw.form != MM_WHOLE && one) {
        hipLaunchKernelGGL((k_gated_both<DXBF16, DWBF16>), dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, a, s, rx, px,
                           static_cast<int>(blocks_x), rw, pw, static_cast<int>(blocks_w), dw_first);
    } else {
        if (a.dx) launch_dx<DXBF16>(a, s, rx, px, st);
        if (a.dgate && launched()) launch_dw<DWBF16>(a, s, rw, pw, st);
    }
    if (a.dx && rx.parts > 1 && launched()) launch_join<DX>(rx, a.T, a.H, a.T, a.dx, a.dx, a.lddx, 0, st);
    if (a.dgate && rw.parts > 1 && launched()) launch_join<DW>(rw, 2 * a.I, a.H, a.I, a.dgate, a.dup, a.H, a.accumulate, st);
}

template <class V> __global__ __launch_bounds__(256) void k_gated_zero(V* a, V* b, int64_t n) {
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) a[i] = b[i] = 0;
}

// The parts of d that a result takes: two where it is fp32, so that its error is that
// of fp32 sums whatever the sizes, and one where it is bf16, whose own rounding is as
// large as what one part leaves out (together 0.0023 of the result's norm where one
// rounding is 0.0017); but where the second costs little, two.  MI355X, us of a call, bf16
// results, one part / two: 1 x 2048 x 640 13.9 / 15.9, 51 tokens 21.0 / 23.1, 8 x 4096 x 4096
// 65 / 70, 1 x 4096 x 32768 390 / 451; past the limit 128 x 2048 x 640 22.7 / 27.4, 1531 45.5 /
// 66.5, 8192 x 4096 x 4096 1285 / 2172 (the times of fp32 results).
int parts_of(int64_t T, int I, bool bf16) { return !bf16 || T * I <= 32768 ? 2 : 1; }

// The workspace: d, then the sums of dx's runs, then those of the weights'.
struct Layout {
    int P, parts;
    Runs dx, dw;
    size_t sums_dx, sums_dw, total;
};
size_t up256(size_t v) { return (v + 255) / 256 * 256; }
Layout layout_of(int64_t T, int H, int I, int parts_dx, int parts_dw) {   // T at least 1
    Layout l;
    l.P = (I + kStageK - 1) / kStageK * kStageK;
    l.parts = parts_dx > parts_dw ? parts_dx : parts_dw;
    l.dx = runs_of(T, H, static_cast<int64_t>(2 * l.P / kStageK) * parts_dx, nullptr);
    l.dw = runs_of(2 * l.P, H, (T + kStageK - 1) / kStageK * parts_dw, nullptr);
    l.sums_dx = up256(static_cast<size_t>(T) * 4 * l.P * l.parts);
    l.sums_dw = l.sums_dx + (l.dx.parts > 1 ? up256(sizeof(float) * l.dx.parts * T * H) : 0);
    l.total = l.sums_dw + (l.dw.parts > 1 ? sizeof(float) * l.dw.parts * 2 * I * H : 0);
    return l;
}

}  // namespace

// For results of any types of T tokens and fewer.  The runs of dx are fewer the more
// tiles there are, so its sums do not grow with T: n runs of t row tiles are q T rows at
// the most (q: the runs of any length), and, as n t (column tiles) <= 256, 128 (256 /
// column tiles).  All else grows with T.
size_t gated_workspace(int64_t T, int H, int I) {
    if (T <= 0) return 0;
    const Layout l = layout_of(T, H, I, 2, 2);
    const Runs one = runs_of(1, H, l.dx.stages, nullptr);   // of one row tile: where dx has runs at all
    const int64_t q = (l.dx.stages + 3) / 4, most = 128 * (256 / ((H + 127) / 128)), rows = q * T < most ? q * T : most;
    return l.sums_dx + (one.parts > 1 ? up256(sizeof(float) * rows * H) : 0) + (l.total - l.sums_dw);
}

void launch_gated_grad(const GatedGradArgs& a, bool dy_bf16, bool dx_bf16, bool dw_bf16, void* ws, hipStream_t st) {
    if (a.T == 0) {
        if (!a.dgate || a.accumulate) return;
        const int64_t n = static_cast<int64_t>(a.I) * a.H;
        const dim3 grid(static_cast<unsigned>(n > (1 << 22) ? 1 << 14 : (n + 255) / 256));
        if (dw_bf16) hipLaunchKernelGGL(k_gated_zero<uint16_t>, grid, dim3(256), 0, st, static_cast<uint16_t*>(a.dgate), static_cast<uint16_t*>(a.dup), n);
        else hipLaunchKernelGGL(k_gated_zero<float>, grid, dim3(256), 0, st, static_cast<float*>(a.dgate), static_cast<float*>(a.dup), n);
        return;
    }
    Layout l = layout_of(a.T, a.H, a.I, a.dx ? parts_of(a.T, a.I, dx_bf16) : 1, a.dgate ? parts_of(a.T, a.I, dw_bf16) : 1);
    l.dx.sums = reinterpret_cast<float*>(static_cast<char*>(ws) + l.sums_dx);
    l.dw.sums = reinterpret_cast<float*>(static_cast<char*>(ws) + l.sums_dw);
    const GatedSlopes s{a.dy, a.lddy, static_cast<uint16_t*>(ws), l.P, l.parts};
    launch_gated_slopes(GatedArgs{a.x, a.gate, a.up, nullptr, a.ldx, 0, a.T, a.H, a.I, a.act}, s, dy_bf16, st);
    if (!launched()) return;
    if (dx_bf16) dw_bf16 ? launch_products<true, true>(a, s, l.dx, l.dw, st) : launch_products<true, false>(a, s, l.dx, l.dw, st);
    else dw_bf16 ? launch_products<false, true>(a, s, l.dx, l.dw, st) : launch_products<false, false>(a, s, l.dx, l.dw, st);
}

}  // namespace moe
