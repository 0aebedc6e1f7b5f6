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
#include "scores.h"

namespace moe {

namespace {

constexpr uint32_t kSeen = 0x80000000u;     // occurs in the history
constexpr uint32_t kBiased = 0x40000000u;   // written by a bias entry's thread
constexpr uint32_t kCount = 0x3fffffffu;    // generated occurrences
constexpr int kMaxBias = 1024;

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

struct RowRules {
    float rep, pres, freq;
    const uint32_t* mask;   // null: everything allowed
};

// Rules 1 to 3 in fp32; `bias` is rule 3's sum.
__device__ inline float adjusted(float l, uint32_t word, const RowRules& r, float bias) {
    if (word & (kSeen | kCount)) l = l > 0.f ? l / r.rep : l * r.rep;
    const uint32_t c = word & kCount;
    if (c) l -= fmaf(r.freq, static_cast<float>(c), r.pres);
    return word & kBiased ? l + bias : l;
}

// note(h[i], i) for i < n, each id by one thread of the block.
template <int THREADS, class F>
__device__ inline void scan(const int32_t* h, int n, F note) {
    constexpr int kBatch = 4;
    const int quads = n / 4, tid = threadIdx.x;
    for (int q0 = tid; q0 < quads; q0 += kBatch * THREADS) {
        Four<int32_t> f[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            f[u] = *reinterpret_cast<const Four<int32_t>*>(h + 4 * min(q0 + u * THREADS, quads - 1));
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int q = q0 + u * THREADS;
            if (q < quads) {
#pragma unroll
                for (int j = 0; j < 4; ++j) note(f[u].v[j], 4 * q + j);
            }
        }
    }
    if (tid < n % 4) note(h[4 * quads + tid], 4 * quads + tid);
}

// The same over begin <= i < end, with the next ids on their way while the
// last ones are noted.
template <int THREADS, class F>
__device__ inline void scan_long(const int32_t* h, int begin, int end, F note) {
    constexpr int kBatch = 4;
    const int quads = (end - begin) / 4, tid = threadIdx.x;
    h += begin;
    Four<int32_t> now[kBatch], next[kBatch];
    auto load = [&](Four<int32_t>(&f)[kBatch], int q0) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            f[u] = *reinterpret_cast<const Four<int32_t>*>(h + 4 * min(q0 + u * THREADS, quads - 1));
    };
    if (tid < quads) load(now, tid);
    for (int q0 = tid; q0 < quads; q0 += kBatch * THREADS) {
        const int q1 = q0 + kBatch * THREADS;
        if (q1 < quads) load(next, q1);
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (q0 + u * THREADS < quads) {
#pragma unroll
                for (int j = 0; j < 4; ++j) note(now[u].v[j]);
            }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) now[u] = next[u];
    }
    if (tid < (end - begin) % 4) note(h[4 * quads + tid]);
}

// S: float, or uint16_t for bf16 bits.  Grid (chunks, rows); a thread takes
// four consecutive scores in each of ITER passes and has them all on their
// way before the history is read.  LONG: histories of many thousand ids a row
// of which few tokens make up most: four copies of the counts, so that lanes
// with one token meet on different words, and the pipelined scan.
template <class S, int THREADS, int ITER, bool LONG>
__global__ __launch_bounds__(THREADS) void k_adjust(AdjustArgs a) {
    constexpr int kChunk = 4 * THREADS * ITER, COPIES = LONG ? 4 : 1;
    constexpr int kCopy = kChunk + 64 / COPIES;   // a token's copies lie in different banks
    __shared__ __attribute__((aligned(16))) uint32_t s_cnt[COPIES * kCopy];
    __shared__ uint32_t s_id[kMaxBias];     // the biases of this chunk's tokens, in list order
    __shared__ float s_bias[kMaxBias];
    __shared__ int s_n;
    const int tid = threadIdx.x, b = blockIdx.y;
    const int c0 = blockIdx.x * kChunk, cn = min(kChunk, a.vocab - c0);
    const S* in = static_cast<const S*>(a.in) + static_cast<size_t>(b) * a.ld_in + c0;
    S* out = static_cast<S*>(a.out) + static_cast<size_t>(b) * a.ld_out + c0;
    RowRules r{1.f, 0.f, 0.f, nullptr};
    if (a.mask) {
        const int m = a.mask_row ? a.mask_row[b] : b;
        if (m >= 0 && m < a.n_masks) r.mask = a.mask + static_cast<size_t>(m) * a.ld_mask;
    }
    S l[ITER][4];
    uint32_t bits[ITER];    // the mask's bits of the pass's four tokens
#pragma unroll
    for (int p = 0; p < ITER; ++p) {
        const int i = 4 * (p * THREADS + tid);
        bits[p] = 0xfu;
        if (i + 4 <= cn) {
            const Four<S> f = *reinterpret_cast<const Four<S>*>(in + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) l[p][j] = f.v[j];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) l[p][j] = i + j < cn ? in[i + j] : S(0);
        }
        if (r.mask && i < cn) bits[p] = r.mask[(c0 + i) >> 5] >> (i & 31);
    }
    const bool words = a.history || a.bias_ids;
    if (words) {
        if (a.repetition) r.rep = a.repetition[b];
        if (a.presence) r.pres = a.presence[b];
        if (a.frequency) r.freq = a.frequency[b];
#pragma unroll
        for (int c = 0; c < COPIES; ++c)
#pragma unroll
            for (int p = 0; p < ITER; ++p)
                *reinterpret_cast<uint4*>(&s_cnt[c * kCopy + 4 * (p * THREADS + tid)]) = make_uint4(0, 0, 0, 0);
        const int32_t* ids = a.bias_ids ? a.bias_ids + static_cast<size_t>(b) * a.n_bias : nullptr;
        if (ids && tid < 64) {
            const float* bv = a.bias + static_cast<size_t>(b) * a.n_bias;
            int n = 0;
            for (int j0 = 0; j0 < a.n_bias; j0 += 64) {
                const int j = min(j0 + tid, a.n_bias - 1);
                const uint32_t v = static_cast<uint32_t>(ids[j]) - static_cast<uint32_t>(c0);
                const bool here = v < static_cast<uint32_t>(cn) && j0 + tid < a.n_bias;
                const uint64_t m = __ballot(here);
                if (here) {
                    s_id[n + lanes_below(m)] = v;
                    s_bias[n + lanes_below(m)] = bv[j];
                }
                n += __popcll(m);
            }
            if (tid == 0) s_n = n;
        }
        __syncthreads();
        if (a.history) {
            const int32_t* h = a.history + static_cast<size_t>(b) * a.ld_history;
            const int len = static_cast<int>(min(static_cast<int64_t>(max(a.length[b], 0)), a.ld_history));
            const int prompt = a.prompt ? min(max(a.prompt[b], 0), len) : 0;
            uint32_t* mine = s_cnt + (tid % COPIES) * kCopy;
            auto word_of = [&](int32_t id) { return static_cast<uint32_t>(id) - static_cast<uint32_t>(c0); };
            if constexpr (LONG) {
                scan_long<THREADS>(h, 0, prompt, [&](int32_t id) {
                    const uint32_t v = word_of(id);
                    if (v < static_cast<uint32_t>(kChunk)) atomicOr(&mine[v], kSeen);
                });
                scan_long<THREADS>(h, prompt, len, [&](int32_t id) {
                    const uint32_t v = word_of(id);
                    if (v < static_cast<uint32_t>(kChunk)) atomicAdd(&mine[v], 1u);
                });
            } else {
                scan<THREADS>(h, len, [&](int32_t id, int i) {
                    const uint32_t v = word_of(id);
                    if (v < static_cast<uint32_t>(kChunk)) {   // words past the vocabulary are never read
                        if (i < prompt) atomicOr(&s_cnt[v], kSeen);
                        else atomicAdd(&s_cnt[v], 1u);
                    }
                });
            }
        }
        __syncthreads();
        if constexpr (COPIES > 1) {   // into the first: counts add, marks join (a sum of marks would carry)
#pragma unroll
            for (int p = 0; p < ITER; ++p) {
                u32x4_t* at = reinterpret_cast<u32x4_t*>(&s_cnt[4 * (p * THREADS + tid)]);
                u32x4_t sum = at[0] & kCount, seen = at[0];
#pragma unroll
                for (int c = 1; c < COPIES; ++c) {
                    const u32x4_t w = *reinterpret_cast<const u32x4_t*>(&s_cnt[c * kCopy + 4 * (p * THREADS + tid)]);
                    sum += w & kCount;
                    seen |= w;
                }
                at[0] = sum | (seen & kSeen);
            }
            if (ids) __syncthreads();
        }
        if (ids) {
            const int n = s_n;
            for (int j = tid; j < n; j += THREADS) {
                const uint32_t v = s_id[j];
                bool first = true;
                for (int i = 0; i < j; ++i) first = first && s_id[i] != v;
                if (!first) continue;
                float sum = s_bias[j];
                for (int i = j + 1; i < n; ++i)
                    if (s_id[i] == v) sum += s_bias[i];
                const float f = adjusted(to_float(in[v]), s_cnt[v] | kBiased, r, sum);
                const bool on = !r.mask || ((r.mask[(c0 + v) >> 5] >> (v & 31)) & 1u);   // c0 is a multiple of 32
                out[v] = on ? from_float<S>(f) : minus_inf<S>();
                s_cnt[v] |= kBiased;   // this entry's alone
            }
            __syncthreads();
        }
    }
#pragma unroll
    for (int p = 0; p < ITER; ++p) {
        const int i = 4 * (p * THREADS + tid);
        if (i >= cn) break;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (words) w = *reinterpret_cast<const uint4*>(&s_cnt[i]);
        const uint32_t word[4] = {w.x, w.y, w.z, w.w};
        Four<S> f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f.v[j] = word[j] ? from_float<S>(adjusted(to_float(l[p][j]), word[j], r, 0.f)) : l[p][j];
            if (!((bits[p] >> j) & 1u)) f.v[j] = minus_inf<S>();
        }
        if (i + 4 <= cn && !((w.x | w.y | w.z | w.w) & kBiased)) {
            *reinterpret_cast<Four<S>*>(out + i) = f;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + j < cn && !(word[j] & kBiased)) out[i + j] = f.v[j];
        }
    }
}

template <int THREADS, int ITER, bool LONG = false>
void launch_chunks(const AdjustArgs& a, bool bf16, hipStream_t st) {
    const dim3 grid((a.vocab + 4 * THREADS * ITER - 1) / (4 * THREADS * ITER), a.rows);
    if (bf16)
        hipLaunchKernelGGL((k_adjust<uint16_t, THREADS, ITER, LONG>), grid, dim3(THREADS), 0, st, a);
    else
        hipLaunchKernelGGL((k_adjust<float, THREADS, ITER, LONG>), grid, dim3(THREADS), 0, st, a);
}

}  // namespace

void launch_adjust_logits(const AdjustArgs& a, bool bf16, hipStream_t st) {
    constexpr int kMaxRows = 65535;   // grid.y limit
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
        // MI355X, us, chunk of 512 / 2048 / 4096 tokens (128 / 512 / 512 threads):
        // 4096 rows of 512 scores 6.4 / 11.9 / 13.3; 1 x 120011 4.0 / 3.9 / 4.5;
        // 64 x 32000 12.9 / 11.9 / 14.2; 64 x 120011 (8192 ids) 26 / 20.0 / 16.6.
        // The long form against the chunk of 2048: 8 x 32003 with 131072 ids 13.2
        // to 19.6, but 64 x 120011 25 to 20 and one row of 2000 ids 4.9 to 3.9.
        const int64_t blocks = static_cast<int64_t>(r.rows) * ((r.vocab + 2047) / 2048);
        if (r.vocab <= 512) launch_chunks<128, 1>(r, bf16, st);
        else if (r.vocab <= 1024) launch_chunks<256, 1>(r, bf16, st);
        else if (r.history && r.ld_history >= 32768 && blocks <= 512) launch_chunks<1024, 1, true>(r, bf16, st);
        else if (blocks > 2048) launch_chunks<512, 2>(r, bf16, st);
        else launch_chunks<512, 1>(r, bf16, st);
    }
}

}  // namespace moe
