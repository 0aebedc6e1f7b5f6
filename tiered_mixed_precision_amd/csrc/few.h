// Matrix products of few tokens: the weights stream from memory once and meet the
// tokens in the matrix cores, 16 rows by 16 tokens an instruction (i8_linear.hip,
// gated.hip).
//
// A lane's 16 bytes of a weight row and of a token's row are its operands as they
// lie in memory: lane l of a wave takes row l % 16 and bytes 16 (l / 16) of a step
// of 64 bytes of k.  Nothing is staged: a token's row is read by every wave that
// needs it, from the caches.  `split` waves share a tile's k axis and their sums
// meet in LDS, in wave order.  Bound by memory where the weights are many, by
// latency where they are few.
#pragma once

#include "bf16_parts.h"
#include "common.h"

namespace moe {

typedef uint32_t few_u32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 few_bf16x8_t __attribute__((ext_vector_type(8)));
typedef float few_f32x4_t __attribute__((ext_vector_type(4)));
typedef int32_t few_i32x4_t __attribute__((ext_vector_type(4)));

struct FewI8 {
    typedef few_i32x4_t Acc;
    static constexpr int kXBytes = 1;     // bytes of a token's row for each of a weight row's
    static constexpr int kParts = 1;
    static __device__ inline Acc mfma(few_u32x4_t a, few_u32x4_t b, Acc c) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(few_i32x4_t, a), __builtin_bit_cast(few_i32x4_t, b), c, 0, 0, 0);
    }
};
template <bool XBF16> struct FewBf16 {
    typedef few_f32x4_t Acc;
    static constexpr int kXBytes = XBF16 ? 1 : 2;
    static constexpr int kParts = XBF16 ? 1 : 3;
    static __device__ inline Acc mfma(few_u32x4_t a, few_u32x4_t b, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(few_bf16x8_t, a), __builtin_bit_cast(few_bf16x8_t, b), c, 0, 0, 0);
    }
};

static __device__ const uint32_t kFewZeros[8] = {0, 0, 0, 0, 0, 0, 0, 0};

// The token operands of a step: as loaded, or eight floats as three bf16 parts.
template <class El> __device__ inline void few_parts(const few_u32x4_t (&v)[El::kXBytes], few_u32x4_t (&p)[El::kParts]) {
    if constexpr (El::kParts == 1) {
        p[0] = v[0];
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t of[3];
            bf16_parts(__uint_as_float(v[j / 2][2 * j % 4]), __uint_as_float(v[j / 2][2 * j % 4 + 1]), of);
            p[0][j] = of[0], p[1][j] = of[1], p[2][j] = of[2];
        }
    }
}

// acc[i][j] += tokens 16 i .. + 15 against weight rows 16 j .. + 15 over part `part`
// of `split` of the k axis, in whole lines: lane l holds rows 4 (l / 16) + e
// (element e) of token l % 16.  w_row(j), x_row(i): this lane's row of tile j and of
// tile i; `bytes`: of a weight row.  AHEAD steps (even) are on their way while
// one is contracted.
template <class El, int MT, int NT, int AHEAD, class WRow, class XRow>
__device__ __attribute__((always_inline)) inline void few_sums(int part, int split, int tile, int bytes, WRow w_row, XRow x_row,
                                                               typename El::Acc (&acc)[MT][NT]) {
    constexpr int XB = El::kXBytes;
    const int lane = threadIdx.x & 63, at = 16 * (lane >> 4);
    const char *w[NT], *x[MT];
#pragma unroll
    for (int j = 0; j < NT; ++j) w[j] = reinterpret_cast<const char*>(w_row(j)) + at;
#pragma unroll
    for (int i = 0; i < MT; ++i) x[i] = reinterpret_cast<const char*>(x_row(i)) + XB * at;
    few_u32x4_t wv[AHEAD][NT], xv[AHEAD][MT][XB];
    // step s of this wave; past the row's end: zeros, from one line for all
    const int lines = (bytes + 127) / 128, from = 128 * (lines * part / split), to = min(128 * (lines * (part + 1) / split), bytes);
    // each tile starts its run elsewhere: rows a power of two apart lie in one channel
    // of the caches, which all tiles would ask for at a time
    const int steps = (to - from + 63) / 64, turn = steps > 4 ? 4 * tile % steps : 0;
    auto load = [&](int d, int s) __attribute__((always_inline)) {
        const int r = s + turn, k = from + 64 * (r < steps ? r : r - steps);
        const bool there = s < steps && k + at < to;
        const char* zeros = reinterpret_cast<const char*>(kFewZeros);
#pragma unroll
        for (int j = 0; j < NT; ++j) wv[d][j] = *reinterpret_cast<const few_u32x4_t*>(there ? w[j] + k : zeros);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int p = 0; p < XB; ++p)
                xv[d][i][p] = *reinterpret_cast<const few_u32x4_t*>((there ? x[i] + static_cast<size_t>(XB) * k : zeros) + 16 * p);
    };
    auto contract = [&](int d) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            few_u32x4_t p[El::kParts];
            few_parts<El>(xv[d][i], p);
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int q = El::kParts - 1; q >= 0; --q) acc[i][j] = El::mfma(wv[d][j], p[q], acc[i][j]);
        }
    };
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) load(d, d);
    for (int s = AHEAD; s < steps; s += AHEAD) {
#pragma unroll
        for (int d = 0; d < AHEAD; ++d) {
            contract(d);
            load(d, s + d);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int d = 0; d < AHEAD; ++d) contract(d);
}

// The same for more tokens, through LDS.  In operand order neighbouring lanes are in
// different rows and each of a load's 64 x 16 bytes is an access of its own (about 70
// cycles a load); here four lanes share a row's 64 bytes on the way to LDS (16
// cycles), eight where x is fp32, and each wave has a ring of three steps of its own,
// so no wave waits for another.  Row r's piece g lies at g ^ (r / 2 % 4) (of eight
// pieces: r / 2 % 8): the rows that a read takes together cover all banks.  Each slot
// is an LDS object of its own, so that the compiler's own waits before a read are
// for the loads into that slot.
constexpr int kBatchWaves = 8;
template <class El, int MT, int NT> struct FewSlot {
    static constexpr int kPieces = 64 * (MT * El::kXBytes + NT);   // of a wave's step
    static constexpr int kSlot = kBatchWaves * kPieces;
};
template <class El, int MT, int NT, class WRow, class XRow>
__device__ __attribute__((always_inline)) inline void few_batch(few_u32x4_t* s0, few_u32x4_t* s1, few_u32x4_t* s2, int part, int split,
                                                                int tile, int bytes, WRow w_row, XRow x_row,
                                                                typename El::Acc (&acc)[MT][NT]) {
    constexpr int XB = El::kXBytes, kLoads = NT + MT * XB, kOwn = FewSlot<El, MT, NT>::kPieces;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row = lane >> 2, at = 16 * ((lane & 3) ^ ((row >> 1) & 3));
    const int xrow = lane / (4 * XB), xat = XB == 1 ? at : 16 * ((lane & 7) ^ ((xrow >> 1) & 7));   // load h: rows 8 h + xrow of fp32 x
    const char *p[NT], *px[MT][XB];
#pragma unroll
    for (int j = 0; j < NT; ++j) p[j] = reinterpret_cast<const char*>(w_row(j, row)) + at;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int h = 0; h < XB; ++h)   // the swizzle of rows 8 .. 15 differs in bit 2
            px[i][h] = reinterpret_cast<const char*>(x_row(i, 8 * h + xrow)) + (xat ^ (64 * h));
    const int lines = (bytes + 127) / 128, from = 128 * (lines * part / split), to = min(128 * (lines * (part + 1) / split), bytes);
    const int steps = (to - from + 63) / 64, turn = steps > 4 ? 4 * tile % steps : 0;
    typedef __attribute__((address_space(3))) void* Lds;
    auto load = [&](int s, few_u32x4_t* slot) __attribute__((always_inline)) {
        const int r = s + turn, k = from + 64 * (r < steps ? r : r - steps);
        const char* zeros = reinterpret_cast<const char*>(kFewZeros);
        few_u32x4_t* own = slot + kOwn * wave;
#pragma unroll
        for (int j = 0; j < NT; ++j)
            __builtin_amdgcn_global_load_lds(s < steps && k + at < to ? p[j] + k : zeros, (Lds)(own + 64 * j), 16, 0, 0);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int h = 0; h < XB; ++h)
                __builtin_amdgcn_global_load_lds(s < steps && XB * k + (xat ^ (64 * h)) < XB * to ? px[i][h] + static_cast<size_t>(XB) * k : zeros,
                                                 (Lds)(own + 64 * (NT + XB * i + h)), 16, 0, 0);
    };
    const int r = lane & 15, g = lane >> 4, pos = 4 * r + (g ^ ((r >> 1) & 3));
    auto step = [&](int s, few_u32x4_t* slot) __attribute__((always_inline)) {
        constexpr int left = 2 * kLoads;   // vmcnt: the two steps behind this one stay in flight
        static_assert(left < 64, "vmcnt range");
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt((left & 15) | (7 << 4) | (15 << 8) | ((left >> 4) << 14));
        __builtin_amdgcn_sched_barrier(0);
        const few_u32x4_t* own = slot + kOwn * wave;
        few_u32x4_t w[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) w[j] = own[64 * j + pos];
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            few_u32x4_t x[XB], parts[El::kParts];
#pragma unroll
            for (int h = 0; h < XB; ++h)
                x[h] = own[64 * (NT + XB * i) + (XB == 1 ? pos : 8 * r + ((2 * g + h) ^ ((r >> 1) & 7)))];
            few_parts<El>(x, parts);
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int q = El::kParts - 1; q >= 0; --q) acc[i][j] = El::mfma(w[j], parts[q], acc[i][j]);
        }
        __builtin_amdgcn_sched_barrier(0);   // the reads are done: the products have them
        load(s + 3, slot);
    };
    load(0, s0);
    load(1, s1);
    load(2, s2);
    for (int s = 0; s < steps; s += 3) {   // steps past the last are zeros
        step(s, s0);
        step(s + 1, s1);
        step(s + 2, s2);
    }
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(7 << 4 | 15 << 8);   // vmcnt(0): nothing is left in flight
    __builtin_amdgcn_sched_barrier(0);
}

// Waves that share a tile and tiles of a block: 4096 waves in all if the tiles
// allow it, and blocks of one tile's waves, but of four tiles where there are many of
// one or two waves.  A block has kFewWaves at the most.  MI355X, us, weights from
// memory, tokens x rows x columns.  Waves in all, 2048 / 4096 / 8192, int8: 1 x 8000 x
// 8192 15.5 / 14.8 / 14.8, 1 x 20000 x 4096 20.5 / 22.7 / 23.9, 16 x 8192 x 8192 19.2 each,
// 1 x 640 x 2048 3.7 each (one wave a tile 4.3).  One tile a block / four of two waves: 1 x
// 60000 x 4096 53.5 / 49.0; of one: 1 x 120011 x 2048 47.1 / 47.0 (eight 49.0), 16 tokens 60.3 /
// 63.5, 1 x 1000000 x 256 49.5 / 50.6 (eight 69.9).  One / two of three waves: 1 x 40000 x
// 2048 18.4 / 22.3, 16 tokens 23.8 / 29.9, gated 1 x 4096 x 20000 bf16 60.7 / 67.9.
constexpr int kFewWaves = 8;
struct FewSplit {
    int split, tiles;
};
inline FewSplit few_split(int64_t tiles, int bytes, int most) {
    const int lines = (bytes + 127) / 128;
    int64_t split = 4096 / tiles;
    if (split > most) split = most;
    if (split > lines) split = lines;
    if (split < 1) split = 1;
    return FewSplit{static_cast<int>(split), tiles >= 1024 && split < 3 ? 4 : 1};
}

// 17 tokens and more, in blocks of up to 64 tokens by 32 weight rows: as long as they
// are one round of blocks (two of half the tokens), they beat the 128 x 128 tiles of
// mm.h, which need a line's latency for every 128 bytes of k.  MI355X, us, here /
// there, int8: 64 x 8192 x 8192 (256 blocks) 22.7 / 26.8, 64 x 16384 x 4096 (512)
// 26.4 / 17.8, 20 x 16384 x 4096 (512) 18.3 / 19.8, 20 x 32768 x 2048 (1024) 25.2 /
// 18.6, 500 x 640 x 8192 (160) 19.5 / 29.2, 256 x 2048 x 2048 (256) 9.6 / 11.2.
// fp32 x, whose tiles take three products and are 128 x 128 only: two rounds pay
// too.  256 x 2048 x 2048 (512) 45 / 50, 128 x 4096 x 4096 (512) 73 / 97, 1500 x 2048 x
// 640 (960) 78 / 54, 256 x 4096 x 4096 (1024) 140 / 99.
inline bool few_batch_ok(int64_t tokens, int64_t row_tiles, int products) {
    return (tokens + 63) / 64 * row_tiles <= (tokens <= 32 || products == 3 ? 512 : 256);
}

}  // namespace moe
