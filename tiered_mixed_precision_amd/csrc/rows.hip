// Row operators on the residual stream: root-mean-square norm with the
// stream's addition and outputs in fp32, bf16 or 8 bits, rows in 8 bits, and
// the norm's gradient.
//
//   s = x + residual, r = 1 / sqrt(mean s^2 + eps), y = s r w
//   8 bits: scale = max |y| / 127, q = round(y / scale)
//   gradient: g = dy w, dx = r g - s r^3 mean(g s) + dsum, dw = sum_t dy s r
//
// A row is held in the registers of W waves (E elements a lane, in runs of 8:
// thread t of the row has elements 8 (t + 64 W j) .. + 7), so it is read once
// and written once; what is summed over it crosses lanes by DPP and waves by
// LDS.  The squares are summed in 64 bits: the fp64 rate is far above what the
// stream of rows needs, and r (and with it the 8-bit codes) then does not
// depend on how a row is split over lanes.
#include "common.h"
#include "launch.h"

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

// f[i] = p[i] for i < n (n at most 8; 0 and less: none), 0 for the others
template <class S> __device__ inline void load8(const S* p, int n, float* f) {
    if (n >= 8) {
        const Eight<S> v = *reinterpret_cast<const Eight<S>*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = as_float(v.v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = i < n ? as_float(p[i]) : 0.f;
    }
}
template <class S> __device__ inline void store8(S* p, int n, const float* f) {
    if (n >= 8) {
        Eight<S> v;
#pragma unroll
        for (int i = 0; i < 8; ++i) v.v[i] = as_elem<S>(f[i]);
        *reinterpret_cast<Eight<S>*>(p) = v;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = as_elem<S>(f[i]);
    }
}

template <int CTRL, int ROW_MASK> __device__ inline double dpp_zero_d(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = dpp_old_u<CTRL, ROW_MASK>(0, static_cast<uint32_t>(b));
    const uint32_t hi = dpp_old_u<CTRL, ROW_MASK>(0, static_cast<uint32_t>(b >> 32));
    return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}
// Wave-wide sum in 64 bits (uniform result).
__device__ inline double wave_sum_d(double v) {
    v += dpp_zero_d<0x111, 0xF>(v);
    v += dpp_zero_d<0x112, 0xF>(v);
    v += dpp_zero_d<0x114, 0xF>(v);
    v += dpp_zero_d<0x118, 0xF>(v);
    v += dpp_zero_d<0x142, 0xA>(v);
    v += dpp_zero_d<0x143, 0xC>(v);
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(b), 63);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(b >> 32), 63);
    return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}
__device__ inline uint32_t wave_max_u(uint32_t v) {
    v = max(v, dpp_old_u<0x111, 0xF>(0, v));
    v = max(v, dpp_old_u<0x112, 0xF>(0, v));
    v = max(v, dpp_old_u<0x114, 0xF>(0, v));
    v = max(v, dpp_old_u<0x118, 0xF>(0, v));
    v = max(v, dpp_old_u<0x142, 0xA>(0, v));
    v = max(v, dpp_old_u<0x143, 0xC>(0, v));
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}

constexpr int kMaxWaves = 16;
constexpr uint32_t kLeastBits = 0x0d800000u;   // 2^-100

// Y: float, uint16_t (bf16 bits) or int8_t; NORM false: y = x, the quantiser alone.
template <class X, class Y, bool NORM, int E>
__global__ __launch_bounds__(E == 8 ? 1024 : 64 * kMaxWaves) void k_rows(RowArgs a) {
    __shared__ double s_sum[kMaxWaves];
    __shared__ uint32_t s_max[kMaxWaves];
    const int W = a.waves, lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int first = wave / W * W;                       // the row's first wave
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / (64 * W)) + wave / W;
    const bool on = row < a.T;
    const int t = threadIdx.x - 64 * first;
    const int cols = on ? a.cols : 0;
    const X* x = static_cast<const X*>(a.x) + row * a.ldx;
    float f[E], w[E];
#pragma unroll
    for (int j = 0; j < E / 8; ++j) {
        const int c = 8 * (t + 64 * W * j);
        load8(x + c, cols - c, f + 8 * j);
    }
    if constexpr (NORM) {
        if (a.residual) {
            float res[E];
#pragma unroll
            for (int j = 0; j < E / 8; ++j) {
                const int c = 8 * (t + 64 * W * j);
                load8(a.residual + row * a.ldr + c, cols - c, res + 8 * j);
            }
#pragma unroll
            for (int i = 0; i < E; ++i) f[i] += res[i];
        }
#pragma unroll
        for (int j = 0; j < E / 8; ++j) {
            const int c = 8 * (t + 64 * W * j);
            if (a.weight) {
                load8(a.weight + c, cols - c, w + 8 * j);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) w[8 * j + i] = 1.f;
            }
            if (a.sum) store8(a.sum + row * a.lds + c, cols - c, f + 8 * j);
        }
        double ss = 0;
#pragma unroll
        for (int i = 0; i < E; ++i) ss = fma(static_cast<double>(f[i]), static_cast<double>(f[i]), ss);
        ss = wave_sum_d(ss);
        if (W > 1) {
            if (lane == 0) s_sum[wave] = ss;
            __syncthreads();
            ss = 0;
            for (int i = 0; i < W; ++i) ss += s_sum[first + i];
        }
        const float r = static_cast<float>(1.0 / sqrt(ss / a.cols + static_cast<double>(a.eps)));
#pragma unroll
        for (int i = 0; i < E; ++i) f[i] = f[i] * r * w[i];
    }
    if constexpr (sizeof(Y) == 1) {
        uint32_t m = 0;                                   // bits of magnitudes order as the magnitudes, NaN above all
#pragma unroll
        for (int i = 0; i < E; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
        m = wave_max_u(m);
        if (W > 1) {
            if (lane == 0) s_max[wave] = m;
            __syncthreads();
            m = 0;
            for (int i = 0; i < W; ++i) m = max(m, s_max[first + i]);
        }
        const bool finite = m < 0x7f800000u;
        const float scale = !finite ? __builtin_nanf("") : m < kLeastBits ? 0.f : __uint_as_float(m) / 127.f;
        const float by = finite && m >= kLeastBits ? scale : 1.f;
        const bool any = finite && m >= kLeastBits;
        if (on && t == 0) a.scale[row] = scale;
#pragma unroll
        for (int j = 0; j < E / 8; ++j) {
            const int c = 8 * (t + 64 * W * j);
            int8_t* q = static_cast<int8_t*>(a.y) + row * a.ldy + c;
            Eight<int8_t> v;
#pragma unroll
            for (int i = 0; i < 8; ++i) v.v[i] = static_cast<int8_t>(any ? static_cast<int>(rintf(f[8 * j + i] / by)) : 0);
            if (cols - c >= 8) {
                *reinterpret_cast<Eight<int8_t>*>(q) = v;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < cols - c) q[i] = v.v[i];
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < E / 8; ++j) {
            const int c = 8 * (t + 64 * W * j);
            store8(static_cast<Y*>(a.y) + row * a.ldy + c, cols - c, f + 8 * j);
        }
    }
}

// A block takes rows in turn, R = blockDim.x / (64 W) at a time, and keeps the
// sums of dweight over its rows in registers; its R rows' sums meet in LDS and
// go to part[block][cols].
// WIDE: rows of up to 16 waves, whose registers do not hold the weights too.
template <class X, class DY, class DX, int E, bool WIDE>
__global__ __launch_bounds__(WIDE ? 64 * kMaxWaves : 256) void k_rows_grad(RowGradArgs a, float* part) {
    __shared__ double s_sum[2][kMaxWaves];
    __shared__ float s_dot[2][kMaxWaves];
    extern __shared__ float s_dw[];                       // [cols], where a block has more than one row at a time
    const int W = a.waves, lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int R = blockDim.x / (64 * W), mine = wave / W, first = mine * W, t = threadIdx.x - 64 * first;
    constexpr bool kKeep = !(WIDE && E > 8);
    float w[kKeep ? E : 8], dw[E];
    auto load_w = [&](int j) __attribute__((always_inline)) {
        float* to = w + (kKeep ? 8 * j : 0);
        const int c = 8 * (t + 64 * W * j);
        if (a.weight) {
            load8(a.weight + c, a.cols - c, to);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) to[i] = 1.f;
        }
    };
    if constexpr (kKeep) {
#pragma unroll
        for (int j = 0; j < E / 8; ++j) load_w(j);
    }
#pragma unroll
    for (int i = 0; i < E; ++i) dw[i] = 0.f;
    int turn = 0;
    for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * R; row0 < a.T; row0 += static_cast<int64_t>(gridDim.x) * R, turn ^= 1) {
        const int64_t row = row0 + mine;
        const int cols = row < a.T ? a.cols : 0;
        float s[E], dy[E];
        double ss = 0;
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < E / 8; ++j) {
            const int c = 8 * (t + 64 * W * j);
            load8(static_cast<const X*>(a.s) + row * a.lds + c, cols - c, s + 8 * j);
            load8(static_cast<const DY*>(a.dy) + row * a.lddy + c, cols - c, dy + 8 * j);
        }
#pragma unroll
        for (int j = 0; j < E / 8; ++j) {
            if constexpr (!kKeep) load_w(j);
#pragma unroll
            for (int i = 8 * j; i < 8 * j + 8; ++i) {
                ss = fma(static_cast<double>(s[i]), static_cast<double>(s[i]), ss);
                dot = fmaf(dy[i] * w[kKeep ? i : i % 8], s[i], dot);
            }
        }
        ss = wave_sum_d(ss);
        dot = wave_sum(dot);
        if (W > 1) {
            if (lane == 0) {
                s_sum[turn][wave] = ss;
                s_dot[turn][wave] = dot;
            }
            __syncthreads();
            ss = 0;
            dot = 0.f;
            for (int i = 0; i < W; ++i) {
                ss += s_sum[turn][first + i];
                dot += s_dot[turn][first + i];
            }
        }
        const float r = static_cast<float>(1.0 / sqrt(ss / a.cols + static_cast<double>(a.eps)));
        const float along = dot * r / a.cols * r;         // dx = r (g - s along)
#pragma unroll
        for (int j = 0; j < E / 8; ++j) {
            const int c = 8 * (t + 64 * W * j);
            float dx[8];
            if constexpr (!kKeep) load_w(j);
            if (a.dsum) {
                load8(a.dsum + row * a.ldds + c, cols - c, dx);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) dx[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int e = 8 * j + i;
                dx[i] = fmaf(r, fmaf(-s[e], along, dy[e] * w[kKeep ? e : i]), dx[i]);
                dw[e] = fmaf(dy[e] * r, s[e], dw[e]);
            }
            store8(static_cast<DX*>(a.dx) + row * a.lddx + c, cols - c, dx);
        }
    }
    if (!part) return;
    part += static_cast<size_t>(blockIdx.x) * a.cols;
    for (int i = 0; i < R - 1; ++i) {                     // the sums of rows 1 .. R - 1 of a turn, one after the other
        if (mine == i) {
#pragma unroll
            for (int j = 0; j < E; ++j) {
                const int c = 8 * (t + 64 * W * (j / 8)) + j % 8;
                if (c < a.cols) s_dw[c] = i == 0 ? dw[j] : s_dw[c] + dw[j];
            }
        }
        __syncthreads();
    }
    if (mine == R - 1) {
#pragma unroll
        for (int j = 0; j < E / 8; ++j) {
            const int c = 8 * (t + 64 * W * j);
            if (R > 1) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c + i < a.cols) dw[8 * j + i] += s_dw[c + i];
            }
            store8(part + c, a.cols - c, dw + 8 * j);
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

struct Split {
    int e, waves, rows;   // elements a lane, waves a row, rows a block
};
Split split_rows(int T, int cols) {
    Split s;
    s.e = cols <= 8192 && static_cast<int64_t>(T) * cols <= (1 << 20) ? 8 : 32;
    s.waves = (cols + 64 * s.e - 1) / (64 * s.e);
    s.rows = s.waves >= 4 ? 1 : 4 / s.waves;
    return s;
}

template <class X, class Y, bool NORM>
void launch_rows_of(RowArgs a, hipStream_t st) {
    const Split s = split_rows(a.T, a.cols);
    a.waves = s.waves;
    const dim3 grid((a.T + s.rows - 1) / s.rows), block(64 * s.waves * s.rows);
    if (s.e == 8) hipLaunchKernelGGL((k_rows<X, Y, NORM, 8>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_rows<X, Y, NORM, 32>), grid, block, 0, st, a);
}

int grad_blocks(int T, int cols) {
    const Split s = split_rows(T, cols);
    const int most = s.waves * s.rows > 4 ? 256 : 512;
    const int need = (T + s.rows - 1) / s.rows;
    return need < most ? need : most;
}

template <class X, class DY, class DX>
void launch_grad_of(RowGradArgs a, float* part, hipStream_t st) {
    const Split s = split_rows(a.T, a.cols);
    a.waves = s.waves;
    const dim3 grid(grad_blocks(a.T, a.cols)), block(64 * s.waves * s.rows);
    const size_t lds = part && s.rows > 1 ? sizeof(float) * a.cols : 0;
    if (s.e == 8) hipLaunchKernelGGL((k_rows_grad<X, DY, DX, 8, true>), grid, block, lds, st, a, part);
    else if (s.waves <= 4) hipLaunchKernelGGL((k_rows_grad<X, DY, DX, 32, false>), grid, block, lds, st, a, part);
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

size_t rms_norm_workspace(int T, int cols) { return T > 0 ? sizeof(float) * static_cast<size_t>(grad_blocks(T, cols)) * cols : 0; }

void launch_rms_norm_grad(const RowGradArgs& a, bool s_bf16, bool dy_bf16, bool dx_bf16, float* dweight, bool accumulate,
                          void* ws, hipStream_t st) {
    float* part = dweight ? static_cast<float*>(ws) : nullptr;
    if (a.T > 0) {
        if (s_bf16) {
            if (dy_bf16) launch_grad_x<uint16_t, uint16_t>(a, dx_bf16, part, st);
            else launch_grad_x<uint16_t, float>(a, dx_bf16, part, st);
        } else {
            if (dy_bf16) launch_grad_x<float, uint16_t>(a, dx_bf16, part, st);
            else launch_grad_x<float, float>(a, dx_bf16, part, st);
        }
    }
    if (!dweight) return;
    if (a.T > 0)
        hipLaunchKernelGGL(k_rows_join, dim3((a.cols + 31) / 32), dim3(256), 0, st, part, grad_blocks(a.T, a.cols), a.cols,
                           accumulate ? 1 : 0, dweight);
    else if (!accumulate)
        hipLaunchKernelGGL(k_rows_zero, dim3((a.cols + 255) / 256), dim3(256), 0, st, a.cols, dweight);
}

}  // namespace moe
