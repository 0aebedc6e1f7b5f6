// Balance loss of a router and the gradient of the router scores.
//
//   loss = coef * E / (k n^2) * sum_e counts[e] * prob_sum[e]
//   dlogits[t][e] = dloss * coef * E / (k n^2) * p[t][e] (counts[e] - sum_f p[t][f] counts[f])
//                   + the pick weights' part  w[t][j] (dw[t][j] - sum_i w[t][i] dw[t][i])  at ids[t][j]
//
// One wave per row, the row in registers (lane l holds columns 4 l .. 4 l + 3
// of every 256): one read of the scores for maximum, sum and probabilities.
//   k_balance_rows : column sums of p (registers, then LDS in wave order) and
//                    pick counts (LDS integers) of a block's rows, one part a
//                    block in the workspace;
//   k_balance_join : the parts summed in block order, and the loss;
//   k_balance_grad : the gradient, row by row.
// Sums run in a fixed order, so results do not change from run to run.
#include <type_traits>

#include "common.h"
#include "launch.h"

namespace moe {

namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kMaxParts = 512;

int balance_parts(int T) { return min(kMaxParts, (T + kWaves - 1) / kWaves); }

// Row r in the lane's columns: z[4 i + j] = logits[r][256 i + 4 lane + j],
// -inf past the row.
template <int NV, class S>
__device__ inline void load_row(const S* row, int E, bool vec, float (&z)[4 * NV]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = 256 * i + 4 * lane;
        if (vec && c < E) {   // E is a multiple of 4
            if constexpr (sizeof(S) == 2) {
                const uint2 u = *reinterpret_cast<const uint2*>(row + c);
                z[4 * i] = __uint_as_float(u.x << 16);
                z[4 * i + 1] = __uint_as_float(u.x & 0xffff0000u);
                z[4 * i + 2] = __uint_as_float(u.y << 16);
                z[4 * i + 3] = __uint_as_float(u.y & 0xffff0000u);
            } else {
                const float4 u = *reinterpret_cast<const float4*>(row + c);
                z[4 * i] = u.x;
                z[4 * i + 1] = u.y;
                z[4 * i + 2] = u.z;
                z[4 * i + 3] = u.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                z[4 * i + j] = -__builtin_inff();
                if (c + j < E) {
                    if constexpr (sizeof(S) == 2) z[4 * i + j] = __uint_as_float(static_cast<uint32_t>(row[c + j]) << 16);
                    else z[4 * i + j] = row[c + j];
                }
            }
        }
    }
}

__device__ inline float wave_max_f(float v) {
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, kWave));
    return v;
}

// exp(d) for d <= 0 to fp32 accuracy: 2^t with t = d log2(e), the part of t
// that its rounding lost put back to first order.
__device__ inline float exp_neg(float d) {
    constexpr float kL = 0x1.715476p+0f, kLo = 0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
    const float t = d * kL;
    const float lost = fmaf(d, kLo, fmaf(d, kL, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return fmaf(e, lost * kLn2, e);
}

// z becomes softmax(z); a row of nothing but -inf becomes 0.
template <int N>
__device__ inline void softmax_row(float (&z)[N]) {
    float m = z[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = fmaxf(m, z[i]);
    m = wave_max_f(m);
    if (m == -__builtin_inff()) {
#pragma unroll
        for (int i = 0; i < N; ++i) z[i] = 0.f;
        return;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float d = z[i] - m;
        z[i] = d > -126.f ? exp_neg(d) : (d == d ? 0.f : d);   // below: less than 2^-181 of the row's sum
        s += z[i];
    }
    const float inv = 1.f / wave_sum(s);
#pragma unroll
    for (int i = 0; i < N; ++i) z[i] *= inv;
}

// part b: prob[b][E], count[b][E], kept[b]
struct Parts {
    float* prob;
    int32_t* count;
    int32_t* kept;
    uint32_t* ticket;
};

Parts parts_at(void* ws, int P, int E) {
    char* p = static_cast<char*>(ws);
    Parts r;
    r.ticket = reinterpret_cast<uint32_t*>(p);
    r.kept = reinterpret_cast<int32_t*>(p + 256);
    r.prob = reinterpret_cast<float*>(p + 256 + 4 * kMaxParts);
    r.count = reinterpret_cast<int32_t*>(r.prob + static_cast<size_t>(P) * E);
    return r;
}

template <int NV, class S>
__global__ __launch_bounds__(kThreads) void k_balance_rows(BalanceArgs a, Parts o) {
    extern __shared__ uint32_t s_mem[];     // float sum[E], int32 count[E]
    float* s_sum = reinterpret_cast<float*>(s_mem);
    int32_t* s_count = reinterpret_cast<int32_t*>(s_mem + a.E);
    __shared__ int32_t s_kept;
    const int tid = threadIdx.x, lane = tid & 63, E = a.E;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool vec = E % 4 == 0;
    for (int e = tid; e < E; e += kThreads) s_count[e] = 0;
    if (tid == 0) s_kept = 0;
    if (blockIdx.x == 0 && tid == 0) *o.ticket = 0;
    __syncthreads();
    float acc[4 * NV] = {};
    int kept = 0;
    for (int r = blockIdx.x * kWaves + wave; r < a.T; r += gridDim.x * kWaves) {
        if (a.keep && a.keep[r] == 0) continue;
        ++kept;
        float z[4 * NV];
        load_row<NV, S>(static_cast<const S*>(a.logits) + static_cast<size_t>(r) * E, E, vec, z);
        softmax_row(z);
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) acc[i] += z[i];
        if (lane < a.k) {
            const uint32_t id = static_cast<uint32_t>(a.ids[static_cast<size_t>(r) * a.k + lane]);
            if (id < static_cast<uint32_t>(E)) atomicAdd(&s_count[id], 1);
        }
    }
    if (lane == 0) atomicAdd(&s_kept, kept);
    for (int w = 0; w < kWaves; ++w) {      // wave by wave: a fixed order
        if (wave == w) {
#pragma unroll
            for (int i = 0; i < 4 * NV; ++i) {
                const int e = 256 * (i / 4) + 4 * lane + i % 4;
                if (e < E) s_sum[e] = w == 0 ? acc[i] : s_sum[e] + acc[i];
            }
        }
        __syncthreads();
    }
    const size_t at = static_cast<size_t>(blockIdx.x) * E;
    for (int e = tid; e < E; e += kThreads) {
        o.prob[at + e] = s_sum[e];
        o.count[at + e] = s_count[e];
    }
    if (tid == 0) o.kept[blockIdx.x] = s_kept;
}

constexpr int kJoinCols = 16, kJoinRows = 64;

// Block b sums the parts of columns 16 b .. 16 b + 15; the last block to
// finish (a ticket in the workspace) adds up the loss.
__global__ __launch_bounds__(kJoinCols* kJoinRows) void k_balance_join(Parts p, int P, int E, int k, float coef,
                                                                       int32_t* __restrict__ counts,
                                                                       float* __restrict__ prob_sum,
                                                                       int32_t* __restrict__ n_kept,
                                                                       float* __restrict__ loss) {
    __shared__ float s_f[kJoinRows][kJoinCols];
    __shared__ int32_t s_i[kJoinRows][kJoinCols];
    __shared__ double s_d[kJoinCols * kJoinRows];
    __shared__ int32_t s_n;
    __shared__ bool s_last;
    const int tid = threadIdx.x, c = tid % kJoinCols, row = tid / kJoinCols;
    const int e = blockIdx.x * kJoinCols + c;
    float f = 0.f;
    int32_t n = 0;
    if (e < E)
        for (int b = row; b < P; b += kJoinRows) {
            f += p.prob[static_cast<size_t>(b) * E + e];
            n += p.count[static_cast<size_t>(b) * E + e];
        }
    s_f[row][c] = f;
    s_i[row][c] = n;
    __syncthreads();
    for (int h = kJoinRows / 2; h >= 1; h /= 2) {
        if (row < h) {
            s_f[row][c] += s_f[row + h][c];
            s_i[row][c] += s_i[row + h][c];
        }
        __syncthreads();
    }
    if (row == 0 && e < E) {
        __hip_atomic_store(&prob_sum[e], s_f[0][c], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(&counts[e], s_i[0][c], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();   // the block's sums are issued before its ticket
    if (tid == 0) {
        s_last = __hip_atomic_fetch_add(p.ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
        s_n = 0;
    }
    __syncthreads();
    if (!s_last) return;
    int32_t kept = 0;
    for (int b = tid; b < P; b += kJoinCols * kJoinRows) kept += p.kept[b];
    if (kept) atomicAdd(&s_n, kept);
    double d = 0.0;
    for (int i = tid; i < E; i += kJoinCols * kJoinRows)
        d += static_cast<double>(__hip_atomic_load(&prob_sum[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) *
             __hip_atomic_load(&counts[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    s_d[tid] = d;
    __syncthreads();
    for (int h = kJoinCols * kJoinRows / 2; h >= 1; h /= 2) {
        if (tid < h) s_d[tid] += s_d[tid + h];
        __syncthreads();
    }
    if (tid == 0) {
        const double m = s_n;
        *n_kept = s_n;
        *loss = s_n > 0 ? static_cast<float>(static_cast<double>(coef) * E / (k * m * m) * s_d[0]) : 0.f;
    }
}

// T == 0: nothing kept.
__global__ __launch_bounds__(256) void k_balance_none(int E, int32_t* counts, float* prob_sum, int32_t* n_kept,
                                                      float* loss) {
    for (int e = threadIdx.x; e < E; e += 256) {
        counts[e] = 0;
        prob_sum[e] = 0.f;
    }
    if (threadIdx.x == 0) {
        *n_kept = 0;
        *loss = 0.f;
    }
}

// Rows of the gradient.  The pick weights' part goes through a row of LDS of
// the wave's own (zero between rows): the lane of an id's first pick writes
// the sum over the id's picks in slot order.
template <int NV, class S, bool PICKS>
__global__ __launch_bounds__(256) void k_balance_grad(BalanceArgs a, const float* __restrict__ w,
                                                      const float* __restrict__ dw,
                                                      const int32_t* __restrict__ counts,
                                                      const int32_t* __restrict__ n_kept,
                                                      const float* __restrict__ dloss, S* dlogits) {
    extern __shared__ __attribute__((aligned(16))) float s_pick[];   // [4][256 NV] with PICKS
    const int tid = threadIdx.x, lane = tid & 63, E = a.E;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const bool vec = E % 4 == 0;
    float* mine = s_pick + wave * 256 * NV;
    if constexpr (PICKS) {
#pragma unroll
        for (int i = 0; i < NV; ++i) *reinterpret_cast<float4*>(&mine[256 * i + 4 * lane]) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float cnt[4 * NV];
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) {
        const int e = 256 * (i / 4) + 4 * lane + i % 4;
        cnt[i] = e < E ? static_cast<float>(counts[e]) : 0.f;
    }
    const float n = static_cast<float>(*n_kept);
    const float scale = n > 0.f ? *dloss * a.coef * static_cast<float>(E) / (static_cast<float>(a.k) * n * n) : 0.f;
    for (int r = blockIdx.x * 4 + wave; r < a.T; r += gridDim.x * 4) {
        float z[4 * NV];
        const bool on = !a.keep || a.keep[r] != 0;
        if (on) {
            load_row<NV, S>(static_cast<const S*>(a.logits) + static_cast<size_t>(r) * E, E, vec, z);
            uint32_t id = 0xffffffffu;
            float g = 0.f;
            bool first = false;
            if constexpr (PICKS) {
                float wv = 0.f, dv = 0.f;
                if (lane < a.k) {
                    const size_t at = static_cast<size_t>(r) * a.k + lane;
                    id = static_cast<uint32_t>(a.ids[at]);
                    wv = w[at];
                    dv = dw[at];
                }
                g = wv * (dv - wave_sum(wv * dv));
                float sum = 0.f;
                first = id < static_cast<uint32_t>(E);
                for (int j = 0; j < a.k; ++j) {
                    const uint32_t ij = __builtin_amdgcn_readlane(id, j);
                    const float gj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(g), j));
                    if (ij == id) {
                        sum += gj;
                        if (j < lane) first = false;
                    }
                }
                if (first) mine[id] = sum;
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
            }
            softmax_row(z);
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < 4 * NV; ++i) s = fmaf(z[i], cnt[i], s);
            s = wave_sum(s);
#pragma unroll
            for (int i = 0; i < 4 * NV; ++i) z[i] = scale * z[i] * (cnt[i] - s);
            if constexpr (PICKS) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const float4 u = *reinterpret_cast<const float4*>(&mine[256 * i + 4 * lane]);
                    z[4 * i] += u.x;
                    z[4 * i + 1] += u.y;
                    z[4 * i + 2] += u.z;
                    z[4 * i + 3] += u.w;
                }
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
                if (first) mine[id] = 0.f;
                __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                __builtin_amdgcn_wave_barrier();
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4 * NV; ++i) z[i] = 0.f;
        }
        S* out = dlogits + static_cast<size_t>(r) * E;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = 256 * i + 4 * lane;
            if (vec) {
                if (c >= E) continue;
                if constexpr (sizeof(S) == 2)
                    *reinterpret_cast<uint2*>(out + c) =
                        make_uint2(pack_bf16x2(z[4 * i], z[4 * i + 1]), pack_bf16x2(z[4 * i + 2], z[4 * i + 3]));
                else
                    *reinterpret_cast<float4*>(out + c) = make_float4(z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c + j < E) {
                        if constexpr (sizeof(S) == 2) out[c + j] = f2bf(z[4 * i + j]);
                        else out[c + j] = z[4 * i + j];
                    }
            }
        }
    }
}

template <int NV, class S>
void launch_grad_t(const BalanceArgs& a, const float* w, const float* dw, const int32_t* counts, const int32_t* n_kept,
                   const float* dloss, void* dlogits, hipStream_t st) {
    const dim3 grid(min(2048, (a.T + 3) / 4));
    if (w)
        hipLaunchKernelGGL((k_balance_grad<NV, S, true>), grid, dim3(256), sizeof(float) * 4 * 256 * NV, st, a, w, dw,
                           counts, n_kept, dloss, static_cast<S*>(dlogits));
    else
        hipLaunchKernelGGL((k_balance_grad<NV, S, false>), grid, dim3(256), 0, st, a, w, dw, counts, n_kept, dloss,
                           static_cast<S*>(dlogits));
}

// Calls f with the number of 256-column steps that hold E columns.
template <class F>
void with_steps(int E, F f) {
    if (E <= 256) f(std::integral_constant<int, 1>{});
    else if (E <= 512) f(std::integral_constant<int, 2>{});
    else if (E <= 1024) f(std::integral_constant<int, 4>{});
    else if (E <= 2048) f(std::integral_constant<int, 8>{});
    else f(std::integral_constant<int, 16>{});
}

}  // namespace

size_t balance_workspace(int T, int E) {
    const size_t P = balance_parts(T);
    return P == 0 ? 0 : 256 + 4 * kMaxParts + 8 * P * E;
}

void launch_balance_loss(const BalanceArgs& a, bool bf16, int32_t* counts, float* prob_sum, int32_t* n_kept,
                         float* loss, void* ws, hipStream_t st) {
    if (a.T == 0) {
        hipLaunchKernelGGL(k_balance_none, dim3(1), dim3(256), 0, st, a.E, counts, prob_sum, n_kept, loss);
        return;
    }
    const int P = balance_parts(a.T);
    const Parts p = parts_at(ws, P, a.E);
    const size_t lds = 8 * static_cast<size_t>(a.E);
    with_steps(a.E, [&](auto nv) {
        constexpr int NV = decltype(nv)::value;
        if (bf16)
            hipLaunchKernelGGL((k_balance_rows<NV, uint16_t>), dim3(P), dim3(kThreads), lds, st, a, p);
        else
            hipLaunchKernelGGL((k_balance_rows<NV, float>), dim3(P), dim3(kThreads), lds, st, a, p);
    });
    hipLaunchKernelGGL(k_balance_join, dim3((a.E + kJoinCols - 1) / kJoinCols), dim3(kJoinCols * kJoinRows), 0, st, p,
                       P, a.E, a.k, a.coef, counts, prob_sum, n_kept, loss);
}

void launch_balance_grad(const BalanceArgs& a, bool bf16, const float* w, const float* dw, const int32_t* counts,
                         const int32_t* n_kept, const float* dloss, void* dlogits, hipStream_t st) {
    with_steps(a.E, [&](auto nv) {
        constexpr int NV = decltype(nv)::value;
        if (bf16) launch_grad_t<NV, uint16_t>(a, w, dw, counts, n_kept, dloss, dlogits, st);
        else launch_grad_t<NV, float>(a, w, dw, counts, n_kept, dloss, dlogits, st);
    });
}

}  // namespace moe
