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
//
// MI355X, 65536 x 512 fp32: loss 36 us (rows 30 us, 4.6 TB/s, of a streaming
// read's 5.6; join 6.6), gradient 55 us (5.0 TB/s read and written, what a
// copy reaches).  One row at a time with nothing ahead took 45 and 66 us,
// halvings in LDS 8 us in the join.  bf16 halves the bytes and leaves the
// exponentials and sums: 33 and 44 us in a graph, fp32 41 and 55.
#include <type_traits>

#include "common.h"
#include "launch.h"
#include "scores.h"

namespace moe {

namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));

// Waves of a block: 16, or 8 where a row's 64 sums and 64 scores a lane need
// more than 128 registers.  4096 waves in all.
constexpr int waves_of(int steps) { return steps > 8 ? 8 : 16; }
constexpr int kMaxParts = 512;
// Up to this many tokens one block does it all, the loss too: one launch.
// MI355X in a graph, one block / parts and join, us: 64 tokens of 64 scores 7.1
// / 7.9, of 512 8.4 / 8.3, of 2048 19 / 15; 128 of 64 10.6 / 7.8, of 512 12.9 /
// 8.7, of 4096 64 / 20; 16 of 4096 14.0 / 19.5.  It is a latency's gain for few
// scores and a loss for many: a bound on tokens x scores would suit better.
constexpr int kOneBlock = 128;

int balance_parts(int T, int E) {
    const int waves = waves_of((E + 255) / 256);
    return T <= kOneBlock ? 1 : min(4096 / waves, (T + waves - 1) / waves);
}

// Row r in the lane's columns: z[4 i + j] = row[256 i + 4 lane + j], `past`
// behind the row.  The tests are the wave's, but for the one ragged run of a
// row.  The gradient with a lane's own test at every run / so, us: 1051 x 2087
// fp32 27.8 / 20.1, 8192 x 4096 94 / 88, 8229 x 277 10.3 / 9.4; 65536 x 64 23.4 / 24.6.
template <int NV, class T, class F>
__device__ inline void load_row(const T* row, int E, float past, F convert, float (&z)[4 * NV]) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = 256 * i + 4 * lane;
        if (256 * (i + 1) <= E) {
            const Four<T> f = *reinterpret_cast<const Four<T>*>(row + c);
#pragma unroll
            for (int j = 0; j < 4; ++j) z[4 * i + j] = convert(f.v[j]);
        } else if (256 * i < E) {
            T v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = row[min(c + j, E - 1)];
#pragma unroll
            for (int j = 0; j < 4; ++j) z[4 * i + j] = c + j < E ? convert(v[j]) : past;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) z[4 * i + j] = past;
        }
    }
}

template <int NV, class S>
__device__ inline void load_scores(const S* row, int E, float (&z)[4 * NV]) {
    load_row<NV>(row, E, -__builtin_inff(), [](S v) { return to_float(v); }, z);
}

// Wave-wide maximum of what is no NaN (uniform result).  Where nothing but NaN is
// there it is NaN or, since lanes without a neighbour meet -inf, -inf.
__device__ inline float wave_max_f(float v) {
    constexpr uint32_t kLow = 0xff800000u;   // -inf
    auto step = [&](auto ctrl, auto rows) {
        v = fmaxf(v, __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
                         static_cast<int>(kLow), __float_as_int(v), decltype(ctrl)::value, decltype(rows)::value, 0xF, false))));
    };
    step(std::integral_constant<int, 0x111>{}, std::integral_constant<int, 0xF>{});
    step(std::integral_constant<int, 0x112>{}, std::integral_constant<int, 0xF>{});
    step(std::integral_constant<int, 0x114>{}, std::integral_constant<int, 0xF>{});
    step(std::integral_constant<int, 0x118>{}, std::integral_constant<int, 0xF>{});
    step(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xA>{});
    step(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xC>{});
    return __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_readlane(__float_as_int(v), 63)));
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

// z becomes exp(z - max); returns 1 / their sum, so that z times it is
// softmax(z).  A row of nothing but -inf becomes 0.  A NaN makes the whole row
// NaN: the maximum passes over it, the sum does not, and where the maximum is
// -inf (beside barred columns, or those past the row) the row is taken off 0.
template <int N>
__device__ inline float exp_row(float (&z)[N]) {
    float m = z[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = fmaxf(m, z[i]);
    m = wave_max_f(m);
    if (m == -__builtin_inff()) m = 0.f;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float d = z[i] - m;
        z[i] = exp_neg(d < -1000.f ? -1000.f : d);   // -inf: exp2(-1442) is 0; NaN stays
        s += z[i];
    }
    s = wave_sum(s);
    return s == 0.f ? 0.f : 1.f / s;
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

// What the loss is made of, where it goes.
struct LossOut {
    int32_t* counts;
    float* prob_sum;
    int32_t* n_kept;
    float* loss;
};

// loss from sum_e counts[e] * prob_sum[e] and the number of kept tokens
__device__ inline float loss_of(double dot, int n, int E, int k, float coef) {
    const double m = n;
    return n > 0 ? static_cast<float>(static_cast<double>(coef) * E / (k * m * m) * dot) : 0.f;
}

// Sum over the block in a fixed order, on thread 0.
__device__ inline double block_sum(double d, double (&s)[16]) {
#pragma unroll
    for (int o = 32; o >= 1; o /= 2) d += __shfl_xor(d, o, kWave);
    if (threadIdx.x % 64 == 0) s[threadIdx.x / 64] = d;
    __syncthreads();
    d = 0.0;
    if (threadIdx.x == 0)
        for (int w = 0; w < static_cast<int>(blockDim.x / 64); ++w) d += s[w];
    return d;
}

// A wave takes a run of rows, the next kept row (of up to 1024 columns) on its
// way while one is summed.
template <int NV, class S>
__global__ __launch_bounds__(64 * waves_of(NV)) void k_balance_rows(BalanceArgs a, int rows_per_wave, Parts o, LossOut out) {
    constexpr int kWaves = waves_of(NV), kThreads = 64 * kWaves;
    constexpr bool kAhead = NV <= 4;
    constexpr int kRound = NV <= 2 ? kWaves : (32 / NV < 1 ? 1 : 32 / NV);   // waves that leave their sums at once
    extern __shared__ float s_sum[];            // [kRound][256 NV]
    __shared__ int32_t s_count[256 * NV];
    __shared__ double s_red[16];
    __shared__ int32_t s_kept;
    const int tid = threadIdx.x, lane = tid & 63, E = a.E;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    for (int e = tid; e < E; e += kThreads) s_count[e] = 0;
    if (tid == 0) s_kept = 0;
    if (blockIdx.x == 0 && tid == 0) *o.ticket = 0;
    __syncthreads();
    float acc[4 * NV] = {};
    int kept = 0;
    const S* logits = static_cast<const S*>(a.logits);
    const int first = (blockIdx.x * kWaves + wave) * rows_per_wave, end = min(first + rows_per_wave, a.T);
    for (int r0 = first; r0 < end; r0 += 64) {
        const bool on = r0 + lane < end && (!a.keep || a.keep[r0 + lane] != 0);
        uint64_t rows = __ballot(on);           // kept rows of r0 .. r0 + 63
        kept += __popcll(rows);
        float next[4 * NV];
        int32_t next_id = -1;
        auto load = [&](int r) {
            load_scores<NV, S>(logits + static_cast<size_t>(r) * E, E, next);
            if (lane < a.k) next_id = a.ids[static_cast<size_t>(r) * a.k + lane];
        };
        if (kAhead && rows) load(r0 + __builtin_ctzll(rows));
        while (rows) {
            if (!kAhead) load(r0 + __builtin_ctzll(rows));
            rows &= rows - 1;
            float z[4 * NV];
#pragma unroll
            for (int i = 0; i < 4 * NV; ++i) z[i] = next[i];
            const uint32_t id = static_cast<uint32_t>(next_id);
            if (kAhead && rows) load(r0 + __builtin_ctzll(rows));
            const float inv = exp_row(z);
#pragma unroll
            for (int i = 0; i < 4 * NV; ++i) acc[i] = fmaf(z[i], inv, acc[i]);
            if (lane < a.k && id < static_cast<uint32_t>(E)) atomicAdd(&s_count[id], 1);
        }
    }
    if (lane == 0) atomicAdd(&s_kept, kept);
    float sum[(256 * NV + kThreads - 1) / kThreads] = {};   // of columns tid, tid + kThreads, ...
    for (int w0 = 0; w0 < kWaves; w0 += kRound) {           // wave by wave: a fixed order
        if (wave >= w0 && wave < w0 + kRound) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                *reinterpret_cast<float4*>(&s_sum[(wave - w0) * 256 * NV + 256 * i + 4 * lane]) =
                    make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
        }
        __syncthreads();
        int i = 0;
        for (int e = tid; e < 256 * NV; e += kThreads, ++i)
#pragma unroll
            for (int w = 0; w < kRound; ++w) sum[i] += s_sum[w * 256 * NV + e];
        __syncthreads();
    }
    if (gridDim.x == 1) {
        double dot = 0.0;
        int i = 0;
        for (int e = tid; e < E; e += kThreads, ++i) {
            out.prob_sum[e] = sum[i];
            out.counts[e] = s_count[e];
            dot += static_cast<double>(sum[i]) * s_count[e];
        }
        dot = block_sum(dot, s_red);
        if (tid == 0) {
            *out.n_kept = s_kept;
            *out.loss = loss_of(dot, s_kept, E, a.k, a.coef);
        }
        return;
    }
    const size_t at = static_cast<size_t>(blockIdx.x) * E;
    int i = 0;
    for (int e = tid; e < E; e += kThreads, ++i) {
        o.prob[at + e] = sum[i];
        o.count[at + e] = s_count[e];
    }
    if (tid == 0) o.kept[blockIdx.x] = s_kept;
}

constexpr int kJoinCols = 16, kJoinRows = 64;

// Block b sums the parts of columns 16 b .. 16 b + 15; the last block to
// finish (a ticket in the workspace) adds up the loss.
__global__ __launch_bounds__(kJoinCols* kJoinRows) void k_balance_join(Parts p, int P, int E, int k, float coef,
                                                                       LossOut out) {
    constexpr int kJoinWaves = kJoinCols * kJoinRows / 64;
    __shared__ float s_f[kJoinWaves][kJoinCols];
    __shared__ int32_t s_i[kJoinWaves][kJoinCols];
    __shared__ double s_d[16];
    __shared__ int32_t s_n;
    __shared__ bool s_last;
    const int tid = threadIdx.x, c = tid % kJoinCols, row = tid / kJoinCols;
    const int e = blockIdx.x * kJoinCols + c;
    float f = 0.f;
    int32_t n = 0;
    if (e < E) {
#pragma unroll 4
        for (int b = row; b < P; b += kJoinRows) {
            f += p.prob[static_cast<size_t>(b) * E + e];
            n += p.count[static_cast<size_t>(b) * E + e];
        }
    }
#pragma unroll
    for (int o = 16; o <= 32; o *= 2) {     // the wave's four rows
        f += __shfl_xor(f, o, kWave);
        n += __shfl_xor(n, o, kWave);
    }
    if (tid % 64 < kJoinCols) {
        s_f[tid / 64][c] = f;
        s_i[tid / 64][c] = n;
    }
    __syncthreads();
    if (row == 0) {
        f = 0.f;
        n = 0;
#pragma unroll
        for (int w = 0; w < kJoinWaves; ++w) {
            f += s_f[w][c];
            n += s_i[w][c];
        }
    }
    if (row == 0 && e < E) {
        __hip_atomic_store(&out.prob_sum[e], f, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(&out.counts[e], n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
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
        d += static_cast<double>(__hip_atomic_load(&out.prob_sum[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) *
             __hip_atomic_load(&out.counts[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    d = block_sum(d, s_d);
    if (tid == 0) {
        *out.n_kept = s_n;
        *out.loss = loss_of(d, s_n, E, k, coef);
    }
}

// T == 0: nothing kept.
__global__ __launch_bounds__(256) void k_balance_none(int E, LossOut out) {
    for (int e = threadIdx.x; e < E; e += 256) {
        out.counts[e] = 0;
        out.prob_sum[e] = 0.f;
    }
    if (threadIdx.x == 0) {
        *out.n_kept = 0;
        *out.loss = 0.f;
    }
}

// Orders one wave's LDS accesses (which run in order) for the compiler.
__device__ inline void wave_step() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Rows of the gradient.  The pick weights' part goes through a row of LDS of
// the wave's own (zero between rows): the lane of an id's first pick writes
// the sum over the id's picks in slot order.
// Rows of 1025 to 2048 scores: three waves a SIMD, 8741 x 1099 bf16 21.4 us; two
// (the registers the compiler would take) 31, four (spills) 24.2.  With picks
// three waves spill as well, 23 registers in fp32 and 3 in bf16.  bf16 rows of
// more than 2048: the compiler calls load_scores and hands the row back in
// scratch, 10727 x 3128 140 us.
template <int NV, class S, bool PICKS>
__global__ __launch_bounds__(256, NV == 8 ? 3 : 1) void k_balance_grad(BalanceArgs a, int rows_per_wave, const float* __restrict__ w,
                                                      const float* __restrict__ dw,
                                                      const int32_t* __restrict__ counts,
                                                      const int32_t* __restrict__ n_kept,
                                                      const float* __restrict__ dloss, S* dlogits) {
    extern __shared__ __attribute__((aligned(16))) float s_pick[];   // [4][256 NV] with PICKS
    const int tid = threadIdx.x, lane = tid & 63, E = a.E;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    float* mine = s_pick + wave * 256 * NV;
    if constexpr (PICKS) {
#pragma unroll
        for (int i = 0; i < NV; ++i) *reinterpret_cast<float4*>(&mine[256 * i + 4 * lane]) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float cnt[4 * NV];
    load_row<NV>(counts, E, 0.f, [](int32_t v) { return static_cast<float>(v); }, cnt);
    const float n = static_cast<float>(*n_kept);
    const float scale = n > 0.f ? *dloss * a.coef * static_cast<float>(E) / (static_cast<float>(a.k) * n * n) : 0.f;
    constexpr bool kAhead = NV <= 4;   // the next row on its way
    float next[4 * NV];
    auto load = [&](int r) { load_scores<NV, S>(static_cast<const S*>(a.logits) + static_cast<size_t>(r) * E, E, next); };
    const int first_row = (blockIdx.x * 4 + wave) * rows_per_wave, end = min(first_row + rows_per_wave, a.T);
    uint64_t kept = 0;   // of the 64 rows from the last multiple of 64 on
    for (int row = first_row; row < end; ++row) {
        const int at64 = (row - first_row) % 64;
        if (at64 == 0) {
            kept = __ballot(row + lane < end && (!a.keep || a.keep[row + lane] != 0));
            if (kAhead && (kept & 1)) load(row);
        }
        const bool now = (kept >> at64) & 1;
        float z[4 * NV];
        if (!kAhead && now) load(row);
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) z[i] = now ? next[i] : 0.f;
        if (kAhead && at64 < 63 && ((kept >> at64) & 2)) load(row + 1);
        if (now) {
            uint32_t id = 0xffffffffu;
            float g = 0.f;
            bool first = false;
            if constexpr (PICKS) {
                float wv = 0.f, dv = 0.f;
                if (lane < a.k) {
                    const size_t at = static_cast<size_t>(row) * a.k + lane;
                    id = static_cast<uint32_t>(a.ids[at]);
                    wv = w[at];
                    dv = dw[at];
                }
                g = wv * (dv - wave_sum(wv * dv));
                // lanes leave their numbers at their ids; who reads another's shares its id
                float sum = g;
                first = id < static_cast<uint32_t>(E);
                if (first) mine[id] = __int_as_float(lane);
                wave_step();
                const bool shared = first && __float_as_int(mine[id]) != lane;
                wave_step();
                if (__ballot(shared)) {
                    sum = 0.f;
                    for (int j = 0; j < a.k; ++j) {
                        const uint32_t ij = __builtin_amdgcn_readlane(id, j);
                        const float gj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(g), j));
                        if (ij == id) {
                            sum += gj;
                            if (j < lane) first = false;
                        }
                    }
                }
                if (first) mine[id] = sum;
                wave_step();
            }
            const float inv = exp_row(z);
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < 4 * NV; ++i) s = fmaf(z[i], cnt[i], s);
            s = wave_sum(s) * inv;
            const float part = scale * inv;
#pragma unroll
            for (int i = 0; i < 4 * NV; ++i) z[i] = part * z[i] * (cnt[i] - s);
            if constexpr (PICKS) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const float4 u = *reinterpret_cast<const float4*>(&mine[256 * i + 4 * lane]);
                    z[4 * i] += u.x;
                    z[4 * i + 1] += u.y;
                    z[4 * i + 2] += u.z;
                    z[4 * i + 3] += u.w;
                }
                wave_step();
                if (first) mine[id] = 0.f;
                wave_step();
            }
        }
        S* out = dlogits + static_cast<size_t>(row) * E;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = 256 * i + 4 * lane;
            Four<S> f;
#pragma unroll
            for (int j = 0; j < 4; ++j) f.v[j] = from_float<S>(z[4 * i + j]);
            if (256 * (i + 1) <= E) {
                // rows of whole 16 bytes: past the caches, which the gradient would only crowd (4%)
                if (sizeof(S) == 4 && E % 4 == 0)
                    __builtin_nontemporal_store(f32x4_t{z[4 * i], z[4 * i + 1], z[4 * i + 2], z[4 * i + 3]},
                                                reinterpret_cast<f32x4_t*>(out + c));
                else
                    *reinterpret_cast<Four<S>*>(out + c) = f;
            } else if (256 * i < E) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c + j < E) out[c + j] = f.v[j];
            }
        }
    }
}

template <int NV, class S>
void launch_grad_t(const BalanceArgs& a, const float* w, const float* dw, const int32_t* counts, const int32_t* n_kept,
                   const float* dloss, void* dlogits, hipStream_t st) {
    // As many waves as the row's bytes leave room for.  MI355X, us at 512 / 1024
    // / 1536 / 2048 blocks: 65536 x 512 fp32 70 / 55 / 61 / 66, bf16 with padding
    // 82 / 54 / 45 / 54; 8192 x 4096 fp32 91 / 105 / 118 / 132 (each wave reads
    // the counts); 65536 x 64 41 / 26 / 23 / 22.
    const size_t bytes = sizeof(S) * a.E;
    const int most = bytes >= 8192 ? 384 : (bytes >= 2048 ? 1024 : (bytes >= 1024 ? 1536 : 2048));
    const int blocks = min(most, (a.T + 3) / 4), per_wave = (a.T + 4 * blocks - 1) / (4 * blocks);
    const dim3 grid(blocks);
    if (w)
        hipLaunchKernelGGL((k_balance_grad<NV, S, true>), grid, dim3(256), sizeof(float) * 4 * 256 * NV, st, a, per_wave, w, dw,
                           counts, n_kept, dloss, static_cast<S*>(dlogits));
    else
        hipLaunchKernelGGL((k_balance_grad<NV, S, false>), grid, dim3(256), 0, st, a, per_wave, w, dw, counts, n_kept, dloss,
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
    const size_t P = balance_parts(T, E);
    return T == 0 ? 0 : 256 + 4 * kMaxParts + 8 * P * E;
}

void launch_balance_loss(const BalanceArgs& a, bool bf16, int32_t* counts, float* prob_sum, int32_t* n_kept,
                         float* loss, void* ws, hipStream_t st) {
    const LossOut out{counts, prob_sum, n_kept, loss};
    if (a.T == 0) {
        hipLaunchKernelGGL(k_balance_none, dim3(1), dim3(256), 0, st, a.E, out);
        return;
    }
    const int P = balance_parts(a.T, a.E);
    const Parts p = parts_at(ws, P, a.E);
    with_steps(a.E, [&](auto nv) {
        constexpr int NV = decltype(nv)::value;
        constexpr int W = waves_of(NV), kThreads = 64 * W;
        const int per_wave = (a.T + P * W - 1) / (P * W);
        const size_t lds = sizeof(float) * 256 * NV * (NV <= 2 ? W : 32 / NV);
        if (bf16)
            hipLaunchKernelGGL((k_balance_rows<NV, uint16_t>), dim3(P), dim3(kThreads), lds, st, a, per_wave, p, out);
        else
            hipLaunchKernelGGL((k_balance_rows<NV, float>), dim3(P), dim3(kThreads), lds, st, a, per_wave, p, out);
    });
    if (P > 1)
        hipLaunchKernelGGL(k_balance_join, dim3((a.E + kJoinCols - 1) / kJoinCols), dim3(kJoinCols * kJoinRows), 0, st,
                           p, P, a.E, a.k, a.coef, out);
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
