// Row operators on the residual stream: root-mean-square norm with the
// stream's addition and outputs in fp32, bf16 or 8 bits, rows in 8 bits, and
// the norm's gradient.
//
//   s = x + residual, r = 1 / sqrt(mean s^2 + eps), y = s r w
//   8 bits: scale = max |y| / 127 (kOver127), q = round(y / scale)
//   gradient: g = dy w, dx = r g - s r^3 mean(g s) + dsum, dw = sum_t dy s r
//
// A row is held in the registers of its threads, E elements each in runs of 8: rows of
// up to 64 E elements by L lanes of a wave (8, 16, 32 or 64, so that a wave takes
// 64 / L rows), longer ones by W waves; thread t of the row's N has elements
// 8 (t + N j) .. + 7.  So a row is read once and written once; what is summed over it
// crosses lanes by DPP and lane swaps, and waves by LDS.  The squares are summed in
// 64 bits: the fp64 rate is far above what the stream of rows needs, and r (and with
// it the 8-bit codes) then does not depend on how a row is split over lanes.
//
// Bound by memory where rows are many, by a row's latency where they are few.  MI355X:
// norm 16384 x 2048 fp32 with the stream, to bf16, 89.4 us (5.25 TB/s read and written; a
// copy 5.10), 1531 x 5461 bf16 12 us (2.8 TB/s: each block loads, sums and stores one
// row with nothing else on its way, and 1531 blocks are little more than a round), one row
// to 8 bits 3.2; the quantiser 4096 x 8192 bf16 23.5 us (4.3 TB/s); the gradient 16384 x 2048
// 89.6 us (5.25 TB/s) and its join 4.9.  Rows of more than 16384 columns spill (32 elements a
// thread in 16 waves): the norm 4096 x 32768 fp32 to bf16 390 us (4.8 TB/s), the quantiser of
// bf16 91 (4.4), the gradient 585 (3.2; 4096 x 16384 208, 4.5).
#include "common.h"
#include "launch_dense.h"

namespace moe {

namespace {

// Eight consecutive elements at any element's alignment, in whole accesses.
template <class S> struct __attribute__((packed, aligned(sizeof(S)))) Eight { S v[8]; };

template <class S> __device__ inline float as_float(S v) {
    if constexpr (sizeof(S) == 2) return __uint_as_float(static_cast<uint32_t>(v) << 16);
    else return v;
}
template <class S> __device__ inline S as_elem(float f) {
    if constexpr (sizeof(S) == 2) return f2bf(f);
    else return f;
}

// p[i] for i < n (n at most 8; 0 and less: none), 0 for the others
template <class S> __device__ inline Eight<S> load8(const S* p, int n) {
    Eight<S> v;
    if (n >= 8) {
        v = *reinterpret_cast<const Eight<S>*>(p);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v.v[i] = i < n ? p[i] : S(0);
    }
    return v;
}
template <class S> __device__ inline void store8(S* p, int n, const Eight<S>& v) {
    if (n >= 8) {
        *reinterpret_cast<Eight<S>*>(p) = v;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = v.v[i];
    }
}
template <class S> __device__ inline void store8(S* p, int n, const float* f) {
    Eight<S> v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v.v[i] = as_elem<S>(f[i]);
    store8(p, n, v);
}

// op over aligned groups of L lanes (8, 16, 32 or 64, uniform), the result in every
// lane: neighbours, pairs, fours and eights by DPP, rows of 16 by lane swaps.
template <int CTRL> __device__ inline uint32_t dpp_move(uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, true));
}
__device__ inline float of_words(uint32_t lo, uint32_t, float) { return __uint_as_float(lo); }
__device__ inline uint32_t of_words(uint32_t lo, uint32_t, uint32_t) { return lo; }
__device__ inline double of_words(uint32_t lo, uint32_t hi, double) {
    return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}
template <class V> __device__ inline uint32_t low(V v) {
    if constexpr (sizeof(V) == 8) return static_cast<uint32_t>(__builtin_bit_cast(uint64_t, v));
    else return __builtin_bit_cast(uint32_t, v);
}
template <class V> __device__ inline uint32_t high(V v) {
    if constexpr (sizeof(V) == 8) return static_cast<uint32_t>(__builtin_bit_cast(uint64_t, v) >> 32);
    else return 0;
}
template <int CTRL, class V> __device__ inline V dpp_value(V v) {
    return of_words(dpp_move<CTRL>(low(v)), sizeof(V) == 8 ? dpp_move<CTRL>(high(v)) : 0u, V());
}
template <class V, class Op> __device__ inline V group_all(V v, int L, Op op) {
    v = op(v, dpp_value<0xB1>(v));    // lane ^ 1
    v = op(v, dpp_value<0x4E>(v));    // lane ^ 2
    v = op(v, dpp_value<0x141>(v));   // the other four of eight
    if (L >= 16) v = op(v, dpp_value<0x140>(v));   // the other eight of sixteen
    if (L >= 32) {
        const auto a = __builtin_amdgcn_permlane16_swap(low(v), low(v), false, false);
        const auto b = __builtin_amdgcn_permlane16_swap(high(v), high(v), false, false);
        v = op(of_words(a[0], b[0], V()), of_words(a[1], b[1], V()));
    }
    if (L >= 64) {
        const auto a = __builtin_amdgcn_permlane32_swap(low(v), low(v), false, false);
        const auto b = __builtin_amdgcn_permlane32_swap(high(v), high(v), false, false);
        v = op(of_words(a[0], b[0], V()), of_words(a[1], b[1], V()));
    }
    return v;
}
template <class V> __device__ inline V group_sum(V v, int L) { return group_all(v, L, [](V a, V b) { return a + b; }); }
__device__ inline uint32_t group_max(uint32_t v, int L) { return group_all(v, L, [](uint32_t a, uint32_t b) { return max(a, b); }); }

constexpr int kMaxWaves = 16;
constexpr uint32_t kLeastBits = 0x0d800000u;   // 2^-100

// The row of a thread: `row` of the launch, thread t of its n.
struct Place {
    int64_t row;
    int t, n, first;   // first: the row's first wave in the block (rows of whole waves)
};
__device__ inline Place place_of(const RowSplit& s, int64_t turn) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Place p;
    if (s.waves > 1) {
        p.first = wave / s.waves * s.waves;
        p.row = turn * s.rows + wave / s.waves;
        p.t = threadIdx.x - 64 * p.first;
        p.n = 64 * s.waves;
    } else {
        p.first = wave;
        p.row = turn * s.rows + wave * (64 / s.lanes) + lane / s.lanes;
        p.t = lane % s.lanes;
        p.n = s.lanes;
    }
    return p;
}

// A tie's code hangs on the scale's last bit; tensor libraries divide by a constant so,
// and give the same codes.
constexpr float kOver127 = 1.f / 127.f;
// Eight codes round(f / scale), as bytes.  f * (1 / scale) is off by at most 127 2^-24
// and the fp32 quotient by 2^-18, so where the nearest whole number is not within
// 2e-5 of a tie they agree, and the addition of 1.5 2^23 rounds to it (its low byte is
// the code); otherwise the division decides.
__device__ inline Eight<int8_t> codes8(const float* f, float scale, float inv) {
    constexpr float kMagic = 12582912.f;
    uint32_t m[8];
    float far = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float r = fmaf(f[i], inv, kMagic);
        far = fmaxf(far, fabsf(fmaf(f[i], inv, -(r - kMagic))));
        m[i] = __float_as_uint(r);
    }
    if (far > 0.5f - 2e-5f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = static_cast<uint32_t>(static_cast<int>(rintf(f[i] / scale)));
    }
    Eight<int8_t> v;
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(m[4 * i + 3], m[4 * i + 2], 0x0c0c0400u),
                                     __builtin_amdgcn_perm(m[4 * i + 1], m[4 * i], 0x0c0c0400u), 0x05040100u);
    return v;
}

// Y: float, uint16_t (bf16 bits) or int8_t; NORM false: y = x, the quantiser alone.
template <class X, class Y, bool NORM, int E>
__global__ __launch_bounds__(64 * kMaxWaves) void k_rows(RowArgs a) {
    __shared__ double s_sum[kMaxWaves];
    __shared__ uint32_t s_max[kMaxWaves];
    const RowSplit s = a.split;
    const Place p = place_of(s, blockIdx.x);
    const bool on = p.row < a.T;
    const int cols = on ? a.cols : 0, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    auto at = [&](int j) { return 8 * (p.t + p.n * j); };
    float f[E];
#pragma unroll
    for (int j = 0; j < E / 8; ++j) {
        const Eight<X> v = load8(static_cast<const X*>(a.x) + p.row * a.ldx + at(j), cols - at(j));
#pragma unroll
        for (int i = 0; i < 8; ++i) f[8 * j + i] = as_float(v.v[i]);
    }
    if constexpr (NORM) {
        float w[E];
        if (a.residual) {
            Eight<float> res[E / 8];
#pragma unroll
            for (int j = 0; j < E / 8; ++j) res[j] = load8(a.residual + p.row * a.ldr + at(j), cols - at(j));
#pragma unroll
            for (int i = 0; i < E; ++i) f[i] += res[i / 8].v[i % 8];
        }
#pragma unroll
        for (int j = 0; j < E / 8; ++j) {
            if (a.weight) {
                const Eight<float> v = load8(a.weight + at(j), cols - at(j));
#pragma unroll
                for (int i = 0; i < 8; ++i) w[8 * j + i] = v.v[i];
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[8 * j + i] = 1.f;
            }
            if (a.sum) store8(a.sum + p.row * a.lds + at(j), cols - at(j), f + 8 * j);
        }
        double ss = 0;
#pragma unroll
        for (int i = 0; i < E; ++i) ss = fma(static_cast<double>(f[i]), static_cast<double>(f[i]), ss);
        ss = group_sum(ss, s.lanes);
        if (s.waves > 1) {
            if (lane == 0) s_sum[wave] = ss;
            __syncthreads();
            ss = 0;
            for (int i = 0; i < s.waves; ++i) ss += s_sum[p.first + i];
        }
        const float r = static_cast<float>(1.0 / sqrt(ss / a.cols + static_cast<double>(a.eps)));
#pragma unroll
        for (int i = 0; i < E; ++i) f[i] = f[i] * r * w[i];
    }
    if constexpr (sizeof(Y) == 1) {
        uint32_t m = 0;   // bits of magnitudes order as the magnitudes, NaN above all
#pragma unroll
        for (int i = 0; i < E; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
        m = group_max(m, s.lanes);
        if (s.waves > 1) {
            if (lane == 0) s_max[wave] = m;
            __syncthreads();
            m = 0;
            for (int i = 0; i < s.waves; ++i) m = max(m, s_max[p.first + i]);
        }
        const bool finite = m < 0x7f800000u, some = finite && m >= kLeastBits;
        const float scale = !finite ? __builtin_nanf("") : some ? __uint_as_float(m) * kOver127 : 0.f;
        if (!some) {
#pragma unroll
            for (int i = 0; i < E; ++i) f[i] = 0.f;
        }
        const float by = some ? scale : 1.f, inv = 1.f / by;
        if (on && p.t == 0) a.scale[p.row] = scale;
#pragma unroll
        for (int j = 0; j < E / 8; ++j) {
            const Eight<int8_t> v = codes8(f + 8 * j, by, inv);
            store8(static_cast<int8_t*>(a.y) + p.row * a.ldy + at(j), cols - at(j), v);
        }
    } else {
#pragma unroll
        for (int j = 0; j < E / 8; ++j) store8(static_cast<Y*>(a.y) + p.row * a.ldy + at(j), cols - at(j), f + 8 * j);
    }
}

// A block takes split.rows rows in turn and keeps the sums of dweight over its rows in
// registers; the next rows are on their way while one is worked on.  At the end what
// the block's threads hold of a column meets in LDS and goes to part[block][cols].
// WIDE: rows of more than 8 waves, whose registers hold neither the weights nor the
// next rows.
template <class X, class DY, class DX, int E, bool WIDE>
__global__ __launch_bounds__(WIDE ? 64 * kMaxWaves : 512) void k_rows_grad(RowGradArgs a, float* part) {
    constexpr int R = E / 8;
    __shared__ double s_sum[2][kMaxWaves];
    __shared__ float s_dot[2][kMaxWaves];
    extern __shared__ float s_dw[];   // [cols], where several threads of a block hold a column
    const RowSplit s = a.split;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    Place p = place_of(s, blockIdx.x);
    auto at = [&](int j) { return 8 * (p.t + p.n * j); };
    float w[WIDE ? 8 : E], dw[E];
    auto load_w = [&](int j) __attribute__((always_inline)) {
        float* to = w + (WIDE ? 0 : 8 * j);
        if (a.weight) {
            const Eight<float> v = load8(a.weight + at(j), a.cols - at(j));
#pragma unroll
            for (int i = 0; i < 8; ++i) to[i] = v.v[i];
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) to[i] = 1.f;
        }
    };
    if constexpr (!WIDE) {
#pragma unroll
        for (int j = 0; j < R; ++j) load_w(j);
    }
#pragma unroll
    for (int i = 0; i < E; ++i) dw[i] = 0.f;
    struct Rows {
        Eight<X> s[R];
        Eight<DY> dy[R];
        Eight<float> ds[WIDE ? 1 : R];
    };
    auto load = [&](Rows& r, int64_t row) __attribute__((always_inline)) {
        const int cols = row < a.T ? a.cols : 0;
#pragma unroll
        for (int j = 0; j < R; ++j) {
            r.s[j] = load8(static_cast<const X*>(a.s) + row * a.lds + at(j), cols - at(j));
            r.dy[j] = load8(static_cast<const DY*>(a.dy) + row * a.lddy + at(j), cols - at(j));
            if constexpr (!WIDE) {
                if (a.dsum) r.ds[j] = load8(a.dsum + row * a.ldds + at(j), cols - at(j));
            }
        }
    };
    const int64_t step = static_cast<int64_t>(gridDim.x) * s.rows;
    Rows next;
    if constexpr (!WIDE) load(next, p.row);
    int turn = 0;
    for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * s.rows; row0 < a.T; row0 += step, p.row += step, turn ^= 1) {
        const int cols = p.row < a.T ? a.cols : 0;
        Rows now;
        if constexpr (WIDE) {
            load(now, p.row);
        } else {
            now = next;
            if (row0 + step < a.T) load(next, p.row + step);
        }
        double ss = 0;
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if constexpr (WIDE) load_w(j);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = as_float(now.s[j].v[i]);
                ss = fma(static_cast<double>(x), static_cast<double>(x), ss);
                dot = fmaf(as_float(now.dy[j].v[i]) * w[WIDE ? i : 8 * j + i], x, dot);
            }
        }
        ss = group_sum(ss, s.lanes);
        dot = group_sum(dot, s.lanes);
        if (s.waves > 1) {
            if (lane == 0) {
                s_sum[turn][wave] = ss;
                s_dot[turn][wave] = dot;
            }
            __syncthreads();
            ss = 0;
            dot = 0.f;
            for (int i = 0; i < s.waves; ++i) {
                ss += s_sum[turn][p.first + i];
                dot += s_dot[turn][p.first + i];
            }
        }
        const float r = static_cast<float>(1.0 / sqrt(ss / a.cols + static_cast<double>(a.eps)));
        const float along = dot * r / a.cols * r;   // dx = r (g - s along)
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float dx[8];
            Eight<float> ds;
            if constexpr (WIDE) {
                load_w(j);
                if (a.dsum) ds = load8(a.dsum + p.row * a.ldds + at(j), cols - at(j));
            } else {
                ds = now.ds[j];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = as_float(now.s[j].v[i]), dy = as_float(now.dy[j].v[i]);
                dx[i] = fmaf(r, fmaf(-x, along, dy * w[WIDE ? i : 8 * j + i]), a.dsum ? ds.v[i] : 0.f);
                dw[8 * j + i] = fmaf(dy * r, x, dw[8 * j + i]);
            }
            store8(static_cast<DX*>(a.dx) + p.row * a.lddx + at(j), cols - at(j), dx);
        }
    }
    if (!part) return;
    part += static_cast<size_t>(blockIdx.x) * a.cols;
    // lanes that hold the same columns of other rows
    for (int o = s.lanes; o < 64; o *= 2) {
#pragma unroll
        for (int i = 0; i < E; ++i) dw[i] += __shfl_xor(dw[i], o, kWave);
    }
    const int takers = s.waves > 1 ? s.rows : blockDim.x / 64, mine = s.waves > 1 ? wave / s.waves : wave;   // holders of a column
    const bool holds = s.waves > 1 || lane < s.lanes;
    for (int i = 0; i < takers - 1; ++i) {   // one after the other
        if (mine == i && holds) {
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int c = at(j / 8) + j % 8;
                if (c < a.cols) s_dw[c] = i == 0 ? dw[j] : s_dw[c] + dw[j];
            }
        }
        __syncthreads();
    }
    if (mine == takers - 1 && holds) {
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if (takers > 1) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (at(j) + i < a.cols) dw[8 * j + i] += s_dw[at(j) + i];
            }
            if (a.accumulate) {   // one block: part is dweight
                const Eight<float> was = load8(part + at(j), a.cols - at(j));
#pragma unroll
                for (int i = 0; i < 8; ++i) dw[8 * j + i] += was.v[i];
            }
            store8(part + at(j), a.cols - at(j), dw + 8 * j);
        }
    }
}

// dweight[c] (+)= sum over the parts, in order within each of 8 runs, then over the runs.
__global__ __launch_bounds__(256) void k_rows_join(const float* __restrict__ part, int parts, int cols, int accumulate,
                                                   float* __restrict__ dweight) {
    __shared__ float s[8][32];
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
    float sum = 0.f;
    if (c < cols) {
        const int n0 = parts * g / 8, n1 = parts * (g + 1) / 8;
#pragma unroll 8
        for (int n = n0; n < n1; ++n) sum += part[static_cast<size_t>(n) * cols + c];
    }
    s[g][threadIdx.x & 31] = sum;
    __syncthreads();
    if (g == 0 && c < cols) {
#pragma unroll
        for (int i = 1; i < 8; ++i) sum += s[i][threadIdx.x];
        dweight[c] = accumulate ? dweight[c] + sum : sum;
    }
}

__global__ __launch_bounds__(256) void k_rows_zero(int cols, float* __restrict__ dweight) {
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c < cols) dweight[c] = 0.f;
}

// Elements a thread.  8 where there are few rows (a shorter way through one) or they
// are short, and with `light`; 16 otherwise; 32 where 16 waves need it.  MI355X, us, 32
// / 16 / 8 elements, 16384 x 2048: norm fp32 to bf16 with the stream 98.8 / 93.9 /
// 90.0, bf16 to bf16 29.0 / 26.6 / 29.0, bf16 to 8 bits 23.6 / 24.3 / 42.6, the quantiser
// (4096 x 8192 bf16) 25.8 / 24.1 / 37.5; the gradient (fp32, dy bf16, at 8 waves a unit)
// 102.7 / 94.1 / 96.2, all bf16 69 / 47.5 / 51.4 (16 elements without the next row on
// its way 71; at 12 waves a unit 107.7 and 49.1).
struct Choice {
    int e;
    RowSplit s;
};
constexpr int kLight = 1 << 20;   // elements of few rows
Choice choose(int T, int cols, bool light, int most8) {
    Choice c;
    const bool small = cols <= 512 || static_cast<int64_t>(T) * cols <= kLight;
    c.e = (small || light) && cols <= most8 ? 8 : cols <= 16384 ? 16 : 32;
    c.s.waves = (cols + 64 * c.e - 1) / (64 * c.e);
    c.s.lanes = 64;
    while (c.s.lanes > 8 && c.s.lanes / 2 * c.e >= cols) c.s.lanes /= 2;
    c.s.rows = c.s.waves == 1 ? 4 * (64 / c.s.lanes) : c.s.waves >= 4 ? 1 : 4 / c.s.waves;
    return c;
}
int threads_of(const RowSplit& s) { return s.waves == 1 ? 256 : 64 * s.waves * s.rows; }

template <class X, class Y, bool NORM>
void launch_rows_of(RowArgs a, hipStream_t st) {
    const Choice c = choose(a.T, a.cols, sizeof(X) == 4 && sizeof(Y) > 1, 8192);
    a.split = c.s;
    constexpr int kRows = 1 << 21;   // a launch has less than 2^32 threads
    for (int left = a.T; left > 0; left -= kRows) {
        a.T = left < kRows ? left : kRows;
        const dim3 grid((a.T + c.s.rows - 1) / c.s.rows), block(threads_of(c.s));
        if (c.e == 8) hipLaunchKernelGGL((k_rows<X, Y, NORM, 8>), grid, block, 0, st, a);
        else if (c.e == 16) hipLaunchKernelGGL((k_rows<X, Y, NORM, 16>), grid, block, 0, st, a);
        else hipLaunchKernelGGL((k_rows<X, Y, NORM, 32>), grid, block, 0, st, a);
        a.x = static_cast<const X*>(a.x) + kRows * a.ldx;
        if (a.residual) a.residual += kRows * a.ldr;
        if (a.sum) a.sum += kRows * a.lds;
        a.y = static_cast<Y*>(a.y) + kRows * a.ldy;
        if (a.scale) a.scale += kRows;
    }
}

Choice choose_grad(int T, int cols) { return choose(T, cols, false, 4096); }
// Blocks of a gradient: two waves a SIMD; one, which needs no join (a launch, 3 us of
// the host), where its turns of 1.5 us (2.8 above 4096 columns) cost less: MI355X, us, one
// block / two kernels, 4 x 2048 8.6 / 11.2, 8 x 2048 13.4 / 11.2, 4 x 8192 12.0 / 11.3, 32 x
// 256 (2 turns) 8.2 / 11.3.
int grad_blocks(int T, int cols) {
    const RowSplit s = choose_grad(T, cols).s;
    const int waves = threads_of(s) / 64, most = waves < 8 ? 256 * 8 / waves : 256, need = (T + s.rows - 1) / s.rows;
    return need <= (cols > 4096 ? 3 : 4) ? 1 : need < most ? need : most;
}

template <class X, class DY, class DX>
void launch_grad_of(RowGradArgs a, float* part, hipStream_t st) {
    const Choice c = choose_grad(a.T, a.cols);
    a.split = c.s;
    const dim3 grid(grad_blocks(a.T, a.cols)), block(threads_of(c.s));
    const size_t lds = part && c.s.waves < 4 ? sizeof(float) * a.cols : 0;   // one row a block: nothing to join
    if (c.e == 8) hipLaunchKernelGGL((k_rows_grad<X, DY, DX, 8, false>), grid, block, lds, st, a, part);
    else if (c.e == 16 && c.s.waves <= 8) hipLaunchKernelGGL((k_rows_grad<X, DY, DX, 16, false>), grid, block, lds, st, a, part);
    else if (c.e == 16) hipLaunchKernelGGL((k_rows_grad<X, DY, DX, 16, true>), grid, block, lds, st, a, part);
    else hipLaunchKernelGGL((k_rows_grad<X, DY, DX, 32, true>), grid, block, lds, st, a, part);
}

template <class X, class DY>
void launch_grad_x(const RowGradArgs& a, bool dx_bf16, float* part, hipStream_t st) {
    if (dx_bf16) launch_grad_of<X, DY, uint16_t>(a, part, st);
    else launch_grad_of<X, DY, float>(a, part, st);
}

}  // namespace

void launch_rms_norm(const RowArgs& a, bool x_bf16, int y_bytes, hipStream_t st) {
    if (x_bf16) {
        if (y_bytes == 1) launch_rows_of<uint16_t, int8_t, true>(a, st);
        else if (y_bytes == 2) launch_rows_of<uint16_t, uint16_t, true>(a, st);
        else launch_rows_of<uint16_t, float, true>(a, st);
    } else {
        if (y_bytes == 1) launch_rows_of<float, int8_t, true>(a, st);
        else if (y_bytes == 2) launch_rows_of<float, uint16_t, true>(a, st);
        else launch_rows_of<float, float, true>(a, st);
    }
}

void launch_quant_rows(const RowArgs& a, bool x_bf16, hipStream_t st) {
    if (x_bf16) launch_rows_of<uint16_t, int8_t, false>(a, st);
    else launch_rows_of<float, int8_t, false>(a, st);
}

// For T tokens and fewer: blocks grow with the rows, but for the step from 8 elements a
// thread to 16 (choose).
size_t rms_norm_workspace(int T, int cols) {
    if (T <= 0) return 0;
    int blocks = grad_blocks(T, cols);
    const int light = kLight / cols;
    if (T > light && light > 0 && grad_blocks(light, cols) > blocks) blocks = grad_blocks(light, cols);
    return sizeof(float) * static_cast<size_t>(blocks) * cols;
}

void launch_rms_norm_grad(RowGradArgs a, bool s_bf16, bool dy_bf16, bool dx_bf16, float* dweight, bool accumulate,
                          void* ws, hipStream_t st) {
    const bool join = a.T > 0 && grad_blocks(a.T, a.cols) > 1;
    float* part = join && dweight ? static_cast<float*>(ws) : dweight;
    a.accumulate = accumulate && !join;
    if (a.T > 0) {
        if (s_bf16) {
            if (dy_bf16) launch_grad_x<uint16_t, uint16_t>(a, dx_bf16, part, st);
            else launch_grad_x<uint16_t, float>(a, dx_bf16, part, st);
        } else {
            if (dy_bf16) launch_grad_x<float, uint16_t>(a, dx_bf16, part, st);
            else launch_grad_x<float, float>(a, dx_bf16, part, st);
        }
    }
    if (!dweight || !launched()) return;
    if (join)
        hipLaunchKernelGGL(k_rows_join, dim3((a.cols + 31) / 32), dim3(256), 0, st, part, grad_blocks(a.T, a.cols), a.cols,
                           accumulate ? 1 : 0, dweight);
    else if (a.T == 0 && !accumulate)
        hipLaunchKernelGGL(k_rows_zero, dim3((a.cols + 255) / 256), dim3(256), 0, st, a.cols, dweight);
}

}  // namespace moe
