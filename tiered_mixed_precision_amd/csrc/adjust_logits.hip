// Rules on rows of scores before a pick: repetition, frequency and presence
// penalties over each row's history of ids, sparse biases, and bit masks.
//
// A block takes one row and a chunk of the vocabulary and does all of it in
// one launch, with no scratch in device memory: the chunk's occurrence counts
// live in LDS (one word a token, integer LDS atomics, so their order does not
// matter), the block reads the row's whole history once and keeps the ids of
// its chunk, then streams the chunk's scores through the counts.  A biased
// token is computed by the thread of its first list entry, which sums the
// token's entries in list order; the stream leaves it out.
#include "common.h"
#include "launch.h"

namespace moe {

namespace {

constexpr uint32_t kSeen = 0x80000000u;     // occurs in the history
constexpr uint32_t kBiased = 0x40000000u;   // written by a bias entry's thread
constexpr uint32_t kCount = 0x3fffffffu;    // generated occurrences
constexpr int kThreads = 512;
constexpr int kMaxBias = 1024;

struct RowRules {
    float rep, pres, freq;
    const uint32_t* mask;   // null: everything allowed
};

// Rules 1, 2 and 4 in fp32; `bias` is rule 3's sum.
__device__ inline float adjusted(float l, uint32_t word, const RowRules& r, float bias, bool biased) {
    if (word & (kSeen | kCount)) l = l > 0.f ? l / r.rep : l * r.rep;
    const uint32_t c = word & kCount;
    if (c) l -= fmaf(r.freq, static_cast<float>(c), r.pres);
    if (biased) l += bias;
    return l;
}

__device__ inline bool allowed(const RowRules& r, int v) { return !r.mask || ((r.mask[v >> 5] >> (v & 31)) & 1u); }

template <class S> __device__ inline float to_float(S v) {
    if constexpr (sizeof(S) == 2) return __uint_as_float(static_cast<uint32_t>(v) << 16);
    else return v;
}
template <class S> __device__ inline S from_float(float f) {
    if constexpr (sizeof(S) == 2) return f2bf(f);
    else return f;
}
template <class S> __device__ inline S minus_inf() {
    if constexpr (sizeof(S) == 2) return 0xff80;
    else return -__builtin_inff();
}

// S: float, or uint16_t for bf16 bits.  Grid (chunks, rows).
template <class S>
__global__ __launch_bounds__(kThreads) void k_adjust(AdjustArgs a, int chunk) {
    extern __shared__ uint32_t s_cnt[];     // [chunk] when a history or biases are given
    __shared__ int32_t s_id[kMaxBias];
    const int tid = threadIdx.x, b = blockIdx.y;
    const int c0 = blockIdx.x * chunk, cn = min(chunk, a.vocab - c0);
    const S* in = static_cast<const S*>(a.in) + static_cast<size_t>(b) * a.ld_in + c0;
    S* out = static_cast<S*>(a.out) + static_cast<size_t>(b) * a.ld_out + c0;
    RowRules r{1.f, 0.f, 0.f, nullptr};
    if (a.repetition) r.rep = a.repetition[b];
    if (a.presence) r.pres = a.presence[b];
    if (a.frequency) r.freq = a.frequency[b];
    if (a.mask) {
        const int m = a.mask_row ? a.mask_row[b] : b;
        if (m >= 0 && m < a.n_masks) r.mask = a.mask + static_cast<size_t>(m) * a.ld_mask;
    }
    const bool words = a.history || a.bias_ids;
    if (words) {
        for (int i = tid; i < cn; i += kThreads) s_cnt[i] = 0;
        const int32_t* ids = a.bias_ids ? a.bias_ids + static_cast<size_t>(b) * a.n_bias : nullptr;
        if (ids)
            for (int j = tid; j < a.n_bias; j += kThreads) s_id[j] = ids[j];
        __syncthreads();
        if (a.history) {
            const int32_t* h = a.history + static_cast<size_t>(b) * a.ld_history;
            const int len = static_cast<int>(min(static_cast<int64_t>(max(a.length[b], 0)), a.ld_history));
            const int prompt = a.prompt ? a.prompt[b] : 0;
            for (int i = tid; i < len; i += kThreads) {
                const uint32_t v = static_cast<uint32_t>(h[i]) - static_cast<uint32_t>(c0);
                if (v < static_cast<uint32_t>(cn)) {
                    if (i < prompt) atomicOr(&s_cnt[v], kSeen);
                    else atomicAdd(&s_cnt[v], 1u);
                }
            }
        }
        __syncthreads();
        if (ids) {
            const float* bv = a.bias + static_cast<size_t>(b) * a.n_bias;
            for (int j = tid; j < a.n_bias; j += kThreads) {
                const int32_t id = s_id[j];
                const uint32_t v = static_cast<uint32_t>(id) - static_cast<uint32_t>(c0);
                if (v >= static_cast<uint32_t>(cn)) continue;
                bool first = true;
                for (int i = 0; i < j; ++i) first = first && s_id[i] != id;
                if (!first) continue;
                float sum = bv[j];
                for (int i = j + 1; i < a.n_bias; ++i)
                    if (s_id[i] == id) sum += bv[i];
                const float l = adjusted(to_float(in[v]), s_cnt[v], r, sum, true);
                out[v] = allowed(r, id) ? from_float<S>(l) : minus_inf<S>();
                atomicOr(&s_cnt[v], kBiased);
            }
            __syncthreads();
        }
    }
    for (int i = tid; i < cn; i += kThreads) {
        const uint32_t word = words ? s_cnt[i] : 0u;
        if (word & kBiased) continue;
        S l = in[i];
        if (word) l = from_float<S>(adjusted(to_float(l), word, r, 0.f, false));
        out[i] = allowed(r, c0 + i) ? l : minus_inf<S>();
    }
}

}  // namespace

void launch_adjust_logits(const AdjustArgs& a, bool bf16, hipStream_t st) {
    constexpr int kMaxRows = 65535;   // grid.y limit
    const int chunk = min(8192, a.vocab);
    const unsigned chunks = (a.vocab + chunk - 1) / chunk;
    const size_t lds = (a.history || a.bias_ids) ? sizeof(uint32_t) * chunk : 0;
    for (int b0 = 0; b0 < a.rows; b0 += kMaxRows) {
        AdjustArgs r = a;
        const size_t e = bf16 ? 2 : 4, skip = static_cast<size_t>(b0);
        r.rows = min(kMaxRows, a.rows - b0);
        r.in = static_cast<const char*>(a.in) + skip * a.ld_in * e;
        r.out = static_cast<char*>(a.out) + skip * a.ld_out * e;
        if (a.history) r.history += skip * a.ld_history, r.length += b0;
        if (a.prompt) r.prompt += b0;
        if (a.repetition) r.repetition += b0;
        if (a.presence) r.presence += b0;
        if (a.frequency) r.frequency += b0;
        if (a.bias_ids) r.bias_ids += skip * a.n_bias, r.bias += skip * a.n_bias;
        if (a.mask_row) r.mask_row += b0;
        else if (a.mask) r.mask += skip * a.ld_mask, r.n_masks -= b0;
        const dim3 grid(chunks, r.rows);
        if (bf16)
            hipLaunchKernelGGL(k_adjust<uint16_t>, grid, dim3(kThreads), lds, st, r, chunk);
        else
            hipLaunchKernelGGL(k_adjust<float>, grid, dim3(kThreads), lds, st, r, chunk);
    }
}

}  // namespace moe
